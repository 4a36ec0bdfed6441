// The paged latent cache: append of new tokens, fork of a batch's rows, compaction of the
// pool, copies of pages.
//
// Append and the page copies are bound by HBM.  Fork and compact move few bytes besides: what
// they cost is the chain from one decision to the next (which pages are shared, which are free,
// who gets them), so one cluster of 16 CTAs makes them all, its phases a hardware barrier
// apart, and a second kernel, launched ahead and waiting, writes the rows or moves the pages with
// the whole GPU.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <atomic>
#include <climits>

#include "mla_cache.cuh"
#include "ptx.cuh"

namespace mla {

namespace {

__device__ __forceinline__ void flag(uint32_t* status, uint32_t bits) {
  if (status && bits) atomicOr(status, bits);
}

__device__ __forceinline__ bool is_page(int v, int num_pages) { return (unsigned)v < (unsigned)num_pages; }

__device__ __forceinline__ int pages_of(int keys, int shift) { return (keys + (1 << shift) - 1) >> shift; }

// ------------------------------------------------------------------ append
// two fp32 values in a 64-bit register: one instruction multiplies or accumulates both
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pair(uint32_t lo, uint32_t hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ f32x2 pair(float lo, float hi) { return pair(__float_as_uint(lo), __float_as_uint(hi)); }
__device__ __forceinline__ float2 both(f32x2 v) {
  uint32_t lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(v));
  return make_float2(__uint_as_float(lo), __uint_as_float(hi));
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

template <typename In>
__device__ __forceinline__ void unpack8(const uint4* v, f32x2 (&x)[4]) {
  if constexpr (sizeof(In) == 2) {
    const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = pair(w[e] << 16, w[e] & 0xffff0000u);
  } else {
    x[0] = pair(v[0].x, v[0].y);
    x[1] = pair(v[0].z, v[0].w);
    x[2] = pair(v[1].x, v[1].y);
    x[3] = pair(v[1].z, v[1].w);
  }
}
template <typename In>
__device__ __forceinline__ void load8(const In* src, f32x2 (&x)[4]) {
  const uint4* s = reinterpret_cast<const uint4*>(src);
  uint4 v[2];
  v[0] = __ldg(s);
  if constexpr (sizeof(In) == 4) v[1] = __ldg(s + 1);
  unpack8<In>(v, x);
}
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }

template <bool E4M3>
__device__ __forceinline__ void store8(uint8_t* dst, const f32x2 (&x)[4]) {
  if constexpr (E4M3) {
    uint32_t w[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(both(x[2 * e]), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(both(x[2 * e + 1]), __NV_SATFINITE, __NV_E4M3);
      w[e] = lo | (hi << 16);
    }
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __nv_bfloat162 h = __float22bfloat162_rn(both(x[e]));
      w[e] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <bool E4M3>
__device__ __forceinline__ void store1(uint8_t* row, int d, float x) {
  if constexpr (E4M3) row[d] = __nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3);
  else reinterpret_cast<__nv_bfloat16*>(row)[d] = __float2bfloat16_rn(x);
}

// The row of token i: the largest b with start[b] <= i (a warp's lanes probe 32 rows at a
// time), -1 when there is none.
__device__ __forceinline__ int row_of_token(const int32_t* start, int B, int i, int lane) {
  int lo = 0, n = B;
  while (true) {
    const int step = (n + 31) / 32, at = lo + lane * step;
    const uint32_t m = __ballot_sync(0xffffffffu, lane * step < n && __ldg(start + at) <= i);
    const int k = __popc(m) - 1;
    if (k < 0) return -1;
    lo += k * step;
    n = min(step, n - k * step);
    if (step == 1) return lo;
  }
}

// c = x / sqrt(mean x^2 + eps) * w, 16 of the 512 dims a lane: the sum, the root and the
// products in fp32, one rounding to the cache's type (e4m3: of c times 1 / descale, at most one
// fp32 rounding from the quotient).  The rope key's pair (a, b) of a lane becomes
// (a cos - b sin, b cos + a sin), rounded the same way.
//
// A run of consecutive tokens to a warp, one wave of warps over all of them.  A token's lookups
// are a chain of dependent loads (row, length, page table) longer than everything else it does:
// lane k runs the chain of token k of up to 32 at once, while the first latents are on their way
// into the warp's ring in shared memory; then token by token, kAhead rows ahead of the one at
// hand, each lane reading back what it copied itself.
// Measured: 65.5k prompt tokens, bf16 into e4m3 pages with norm and rotation, 27.1 us (130 MB,
// 4.8 TB/s; a warp to a token 31.8, four tokens held in a warp's registers 28 to 36 over the
// occupancies).  What is left over the 19.2 us of its bytes is the start of the one wave (3 us of
// lookups) and its instructions (52% of the issue slots, beside 45% of HBM).  64 tokens of a
// decode step: 3.2 us, the chain.
constexpr int kAppendThreads = 256, kAppendWarps = kAppendThreads / 32, kAppendWave = 4;

template <typename In, bool E4M3>
__global__ void __launch_bounds__(kAppendThreads, kAppendWave) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int es = E4M3 ? 1 : 2;
  constexpr int kVec = sizeof(In) == 2 ? 1 : 2;    // 16-byte words of 8 values
  constexpr int kAhead = sizeof(In) == 2 ? 4 : 2;  // 32 KB of rings a block either way
  __shared__ uint4 s_ring[kAppendWarps][kAhead][2 * kVec][32];
  const int lane = threadIdx.x & 31;
  uint4(&ring)[kAhead][2 * kVec][32] = s_ring[threadIdx.x >> 5];
  int end = p.num_tokens;
  if (p.token_start) end = min(end, __ldg(p.token_start + p.B));  // behind it is padding
  const int warps = gridDim.x * kAppendWarps, run = (end + warps - 1) / warps;
  const int first = (int)min((long long)end, (long long)(blockIdx.x * kAppendWarps + (threadIdx.x >> 5)) * run);
  const int last = min(end, first + run);
  const int da = p.interleaved ? 2 * lane : lane, db = p.interleaved ? 2 * lane + 1 : lane + 32;
  const In* x = static_cast<const In*>(p.c_new) + 8 * lane;
  const In* y = static_cast<const In*>(p.kpe_new);
  for (int base = first; base < last; base += 32) {
    const int n = min(32, last - base);
    auto fetch = [&](int k) {  // token k's latents into its place in the ring
      if (k < n) {
        const In* row = x + (size_t)(base + k) * p.c_stride;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int q = 0; q < kVec; ++q)
            cp_async16(smem_addr(&ring[k % kAhead][kVec * h + q][lane]), reinterpret_cast<const uint4*>(row + 256 * h) + q);
      }
      cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k < kAhead; ++k) fetch(k);
    // lane k: the slot and position of token k; slot -1: not written
    long long slot = -1;
    int gpos = 0, b = 0;
    if (p.token_start) b = max(row_of_token(p.token_start, p.B, base, lane), 0);
    if (lane < n) {
      const int i = base + lane;
      int nb = p.per_row, k = 0;
      if (p.token_start) {
        int s = __ldg(p.token_start + b), e = __ldg(p.token_start + b + 1);
        while (i >= e && b + 1 < p.B) {
          ++b;
          s = e;
          e = __ldg(p.token_start + b + 1);
        }
        nb = e - s;
        k = i - s;
      } else {
        b = i / p.per_row;
        k = i - b * p.per_row;
      }
      if (k >= 0 && k < nb) {
        gpos = (p.cp_world > 1 ? p.global_seq_lens[b] : p.seq_lens[b]) - nb + k;
        // under context parallelism another rank's key is not written here
        const bool here = p.cp_world <= 1 || gpos < 0 || (gpos / p.cp_interleave) % p.cp_world == p.cp_rank;
        const int pos = dcp_local_bound(gpos, p.cp_world, p.cp_rank, p.cp_interleave), lp = pos >> p.page_shift;
        if (p.kept && (gpos < 0 || pos < p.kept[b])) {  // its row could not grow: those keys are not new
          if (here) flag(p.status, kErrNoPages);
        } else if (gpos < 0 || lp >= p.stride || (p.rope_table && gpos >= p.rope_positions)) {
          if (here) flag(p.status, kErrBadLength);
        } else if (here) {
          const int page = __ldg(p.page_table + (size_t)b * p.stride + lp);
          if (is_page(page, p.num_pages)) slot = ((long long)page << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
          else flag(p.status, kErrBadPage);
        }
      }
    }
    // a token's rope key and angles: a token ahead, in registers
    In na, nb;
    float nc = 1.f, ns = 0.f;
    auto fetch_rope = [&](int k) {
      const int g = __shfl_sync(0xffffffffu, gpos, k);
      const In* row = y + (size_t)(base + k) * p.kpe_stride;
      na = row[da];
      nb = row[db];
      if (p.rope_table && __shfl_sync(0xffffffffu, slot, k) >= 0) {
        nc = __ldg(p.rope_table + (size_t)g * kDRope + lane);
        ns = __ldg(p.rope_table + (size_t)g * kDRope + 32 + lane);
      }
    };
    fetch_rope(0);
    for (int k = 0; k < n; ++k) {
      float a = to_f32(na), c = to_f32(nb);
      const float co = nc, si = ns;
      const long long to = __shfl_sync(0xffffffffu, slot, k);
      if (k + 1 < n) fetch_rope(k + 1);
      cp_async_wait<kAhead - 1>();
      f32x2 v[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint4 w[kVec];
#pragma unroll
        for (int q = 0; q < kVec; ++q) w[q] = ring[k % kAhead][kVec * h + q][lane];
        unpack8<In>(w, v[h]);
      }
      fetch(k + kAhead);
      float scale = p.inv_descale;
      if (p.norm_weight) {
        f32x2 s2 = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) s2 = fma2(v[h][e], v[h][e], s2);
        float s = both(s2).x + both(s2).y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        scale *= rsqrtf(s * (1.f / kDLatent) + p.norm_eps);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          f32x2 g[4];
          load8(static_cast<const In*>(p.norm_weight) + 256 * h + 8 * lane, g);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[h][e] = mul2(v[h][e], g[e]);
        }
      }
      if (E4M3 || p.norm_weight) {  // a bf16 cache's scale is 1
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) v[h][e] = mul2(v[h][e], pair(scale, scale));
      }
      if (p.rope_table) {
        const float a2 = a * co - c * si, c2 = c * co + a * si;
        a = a2;
        c = c2;
      }
      if constexpr (E4M3) {
        a *= p.inv_descale;
        c *= p.inv_descale;
      }
      if (to >= 0) {
        uint8_t* crow = p.ckv + (size_t)to * kDLatent * es;
        store8<E4M3>(crow + 8 * lane * es, v[0]);
        store8<E4M3>(crow + (256 + 8 * lane) * es, v[1]);
        uint8_t* krow = p.kpe + (size_t)to * kDRope * es;
        store1<E4M3>(krow, da, a);
        store1<E4M3>(krow, db, c);
      }
    }
    cp_async_wait<0>();
  }
}

// ------------------------------------------------------------------ page copies
// Units [u0, u1) of the first `slots` keys of a page, latents then rope keys, by nt threads.
__device__ __forceinline__ void copy_slots(const uint8_t* ckv_src, const uint8_t* kpe_src, uint8_t* ckv, uint8_t* kpe,
                                           size_t from, size_t to, int page_shift, int es, int u0, int u1, int slots,
                                           int t, int nt) {
  const int uc = slots * (kDLatent * es / 16);
  const size_t cb = ((size_t)kDLatent * es) << page_shift, kb = ((size_t)kDRope * es) << page_shift;
  const uint4* cs = reinterpret_cast<const uint4*>(ckv_src + from * cb);
  const uint4* ks = reinterpret_cast<const uint4*>(kpe_src + from * kb);
  uint4* cd = reinterpret_cast<uint4*>(ckv + to * cb);
  uint4* kd = reinterpret_cast<uint4*>(kpe + to * kb);
  constexpr int kU = 8;
  for (int base = u0 + t; base < u1; base += kU * nt) {
    uint4 v[kU];
#pragma unroll
    for (int q = 0; q < kU; ++q) {
      const int u = base + q * nt;
      if (u < u1) v[q] = u < uc ? __ldcs(cs + u) : __ldcs(ks + (u - uc));
    }
#pragma unroll
    for (int q = 0; q < kU; ++q) {
      const int u = base + q * nt;
      if (u < u1) {
        if (u < uc) cd[u] = v[q];
        else kd[u - uc] = v[q];
      }
    }
  }
}

// Whole pages, bound by HBM.  A page's latents are 2^k runs of 256 16-byte units and its rope
// keys as many runs of 32, whatever its size and type: a warp takes a run of each at a time,
// nine loads a lane, no lane idle.  Measured on the GB300 (copy rate 6.79 TB/s): 1.2 GB of
// pages moved 302 MB in 48.3 us (6.3 TB/s, 64-key fp8 pages), 604 MB in 91.9 us (6.6 TB/s,
// 64-key bf16), 302 MB in 49.4 us (8-key fp8); runs of 2048 units by a block of 256 threads took
// 53.8, 99.4 and 80.4, bulk copies through shared memory 55.3, 99.6 and 135.
constexpr int kCopyThreads = 256;
constexpr int kCopyWarps = kCopyThreads / 32;
// Blocks to an SM: far more than run at once, so that none ends a wave behind the others
// (4, 16 and 64: 52.5, 48.5 and 48.3 us for the first of the above); 16 where the kernel, not the
// host, knows how many pages there are.
constexpr int kCopyWave = 64, kMoveWave = 16;

__host__ __device__ inline int runs_shift(int page_shift, int es) { return page_shift - 3 + (es == 2 ? 1 : 0); }

__device__ __forceinline__ void copy_pages(const uint8_t* ckv_src, const uint8_t* kpe_src, uint8_t* ckv, uint8_t* kpe,
                                           const int32_t* src, const int32_t* dst, int n, int src_pages, int dst_pages,
                                           int page_shift, int es, uint32_t* status) {
  const int lane = threadIdx.x & 31, sh = runs_shift(page_shift, es);
  const long long items = (long long)n << sh, step = (long long)gridDim.x * kCopyWarps;
  long long it = (long long)blockIdx.x * kCopyWarps + (threadIdx.x >> 5);
  if (it >= items) return;
  int s = __ldcg(src + (it >> sh)), d = __ldcg(dst + (it >> sh));
  while (true) {
    const int run = (int)(it & ((1ll << sh) - 1));
    const bool ok = is_page(s, src_pages) && is_page(d, dst_pages);
    const size_t from = ((size_t)(unsigned)s << sh) + run, to = ((size_t)(unsigned)d << sh) + run;
    const uint4* cs = reinterpret_cast<const uint4*>(ckv_src) + (from << 8) + lane;
    const uint4* ks = reinterpret_cast<const uint4*>(kpe_src) + (from << 5) + lane;
    uint4 v[9];
    if (ok) {
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = __ldcs(cs + 32 * q);
      v[8] = __ldcs(ks);
    } else if (lane == 0) {
      flag(status, kErrBadPage);
    }
    it += step;
    if (it < items) {  // the next run's pages while this one's bytes arrive
      s = __ldcg(src + (it >> sh));
      d = __ldcg(dst + (it >> sh));
    }
    if (ok) {
      uint4* cd = reinterpret_cast<uint4*>(ckv) + (to << 8) + lane;
#pragma unroll
      for (int q = 0; q < 8; ++q) __stcs(cd + 32 * q, v[q]);
      __stcs(reinterpret_cast<uint4*>(kpe) + (to << 5) + lane, v[8]);
    }
    if (it >= items) return;
  }
}

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ CopyParams p) {
  copy_pages(p.ckv_src, p.kpe_src, p.ckv, p.kpe, p.src, p.dst, p.n, p.src_pages, p.dst_pages, p.page_shift, p.es,
             p.status);
}

// ------------------------------------------------------------------ planning: shared pieces
// The sums x of the block's warps (the same in a warp's lanes): x becomes the sum of the warps
// before this one, total the sum of all.  part: 32 ints nobody else uses.
__device__ __forceinline__ void warp_sums(int& x, int* part, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) part[warp] = x;
  __syncthreads();
  const int v = part[lane];
  total = __reduce_add_sync(0xffffffffu, v);
  x = __reduce_add_sync(0xffffffffu, lane < warp ? v : 0);
}

// exclusive prefix of v over the warp's lanes
__device__ __forceinline__ int lane_prefix(int v) {
  const int lane = threadIdx.x & 31;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x - v;
}

// This warp's share of the pool's 32-page words: contiguous, in order of (CTA, warp).
__device__ __forceinline__ void my_words(int num_pages, uint32_t rank, int warp, int& w0, int& w1) {
  const int words = (num_pages + 31) / 32;
  const int per = (words + kPlanCtas * (kPlanThreads / 32) - 1) / (kPlanCtas * (kPlanThreads / 32));
  w0 = min(words, ((int)rank * (kPlanThreads / 32) + warp) * per);
  w1 = min(words, w0 + per);
}

// Bits of this warp's words: test(counts[x]) of its pages x.  The first 32 stay in its lanes
// (`mine`), the others go to memory; returns how many are set.  Eight words' counts are loaded
// before any is tested.
template <typename T>
__device__ __forceinline__ int scan_words(const int32_t* counts, int num_pages, int w0, int w1, uint32_t* words,
                                          uint32_t& mine, T test) {
  const int lane = threadIdx.x & 31;
  int n = 0;
  mine = 0;
  constexpr int kU = 8;
  for (int base = w0; base < w1; base += kU) {
    int v[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int x = 32 * (base + u) + lane;
      v[u] = base + u < w1 && x < num_pages ? __ldcg(counts + x) : 0;
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int w = base + u;
      if (w >= w1) break;
      const uint32_t m = __ballot_sync(0xffffffffu, 32 * w + lane < num_pages && test(v[u]));
      if (w - w0 == lane) mine = m;
      if (w - w0 >= 32 && lane == 0) words[w] = m;
      n += __popc(m);
    }
  }
  return n;
}
// word w of the warp's (all lanes)
__device__ __forceinline__ uint32_t word_of(const uint32_t* words, uint32_t mine, int w0, int w) {
  return w - w0 < 32 ? __shfl_sync(0xffffffffu, mine, w - w0) : __ldcg(words + w);
}

// A CTA's sums to every CTA of the cluster (before a cluster barrier), and after it the sums of
// the CTAs before this one and of all.
__device__ __forceinline__ void publish(int2* sums, uint32_t rank, int x, int y) {
  if (threadIdx.x < kPlanCtas) {
    const uint32_t at = map_to_rank(smem_addr(sums + rank), threadIdx.x);
    st_shared_cluster(at, (uint32_t)x);
    st_shared_cluster(at + 4, (uint32_t)y);
  }
}
__device__ __forceinline__ void collect(const int2* sums, uint32_t rank, int2& before, int2& all) {
  before = all = make_int2(0, 0);
#pragma unroll
  for (int r = 0; r < kPlanCtas; ++r) {
    const int2 s = sums[r];
    if (r < (int)rank) {
      before.x += s.x;
      before.y += s.y;
    }
    all.x += s.x;
    all.y += s.y;
  }
}

// ------------------------------------------------------------------ fork
struct Kin {
  int have, want, keep;
};

// lengths of an output row whose parent holds `have` keys; a change the table cannot hold is
// flagged and not made
__device__ __forceinline__ Kin row_lengths(const ForkParams& p, int have, int i, uint32_t& err) {
  Kin k;
  k.have = have;
  const long long want = (long long)have + (p.add ? p.add[i] : 0);
  if (want < 0 || want > ((long long)p.stride << p.page_shift)) {
    err |= kErrBadLength;
    k.want = have;
  } else {
    k.want = (int)want;
  }
  k.keep = min(have, k.want);
  return k;
}

// Pages [pages of the sinks, drop_end) of a row that keeps `keep` keys lie wholly past the
// sinks and behind every window from here on: the token at position keep sees the keys from
// keep - window_left.
__device__ __forceinline__ int drop_end(const ForkParams& p, int keep) {
  return p.window_left < 0 ? 0 : max(keep - p.window_left, 0) >> p.page_shift;
}

__device__ __forceinline__ int row_len(const ForkParams& p, int b, uint32_t& err) {
  const int K = p.lens[b], cap = p.stride << p.page_shift;
  if (K < 0 || K > cap) err |= kErrBadLength;
  return min(max(K, 0), cap);
}

__device__ __forceinline__ int parent_of(const ForkParams& p, int i, uint32_t& err) {
  const int b = p.parents[i];
  if (b < -1 || b >= p.B) {
    err |= kErrBadRow;
    return -1;
  }
  return b;
}

// The children of an input row: how many rows continue it (c), how many of them write on in
// its last page (g), the lowest of those; and what follows for the counts.
struct alignas(16) Kids {
  int32_t c, g, first, kind;
};
// No child gives keys up, so all of them keep the same pages: a count changes by c - 1, the
// last page's, where g rows write on, by c - g - 1.
constexpr int kSame = 0;    // nobody else holds the last page: who writes on in it is known at once
constexpr int kClaims = 1;  // others hold it, or may: the writers claim it
constexpr int kMixed = 2;   // some child gives keys up: counts go row by row, writers claim

// A row's claim on a page, in the page's count: below every count a caller keeps.
__device__ __forceinline__ int claim_of(int row) { return INT_MIN + row; }
__device__ __forceinline__ bool is_claim(int count) { return count < INT_MIN + kMaxCacheRows; }

// One cluster plans the whole step.  Phases, a cluster barrier between them:
//   0  children of every input row
//   1  counts: per input row where its children are alike (a plain decode step changes none),
//      else +1 for every page an output row shares and -1 for every page its parent held;
//      where nobody claims a page, which rows copy
//   2  (only if there are claims) a page a row is about to write that nobody shares goes to the
//      claimants' lowest row: atomicMin of claim_of(row); after one more barrier who won
//   3  the fresh pages each row needs, free pages counted
//   4  each row's place in the free list, and the list (free pages in ascending order)
// All sums are integer sums and minima: the result does not depend on their order.
// Measured, with the kernel after it: 128 rows over 16384 pages, most going on, 8.9 us, of which
// the phases' round trips to L2 (0.5 us each) and three barriers (0.6 to 0.9 us with the writes
// they wait for) are 7; 256 beams over 65536 pages 12.8 us (on 8 CTAs 14.7 and more: the
// scattered count updates and the scan of the counts go by the SM).
__global__ void __launch_bounds__(kPlanThreads, 1) fork_plan_kernel(const __grid_constant__ ForkParams p) {
  __shared__ Kids s_kids[kPlanThreads];
  __shared__ int part[2][32], s_claims[kPlanCtas];
  __shared__ int2 s_sums[kPlanCtas];
  const uint32_t rank = cluster_ctarank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const CacheWs L = cache_ws(p.num_pages, p.stride, p.ws_rows);
  ForkRow* info = reinterpret_cast<ForkRow*>(p.ws + L.rows);
  uint32_t* words = reinterpret_cast<uint32_t*>(p.ws + L.words);
  int32_t* list = reinterpret_cast<int32_t*>(p.ws + L.list);
  int32_t* stage = reinterpret_cast<int32_t*>(p.ws + L.stage);
  const bool in_place = p.table == p.table_out;
  const int in_page = (1 << p.page_shift) - 1;
  uint32_t err = 0;
  grid_launch_dependents();

  // 0: this CTA's input rows [b0, b0 + nb) and output rows [i0, i0 + ni), one of each to a
  // thread.  What a thread reads for them, and for its share of the children, goes out level by
  // level (a round trip each): parents and lengths, parents' lengths, last pages, their counts.
  static_assert(kMaxCacheRows == kPlanCtas * kPlanThreads, "one row to a thread");
  const int bper = (p.B + kPlanCtas - 1) / kPlanCtas, b0 = min(p.B, (int)rank * bper), nb = min(p.B - b0, bper);
  const int iper = (p.N + kPlanCtas - 1) / kPlanCtas, i0 = min(p.N, (int)rank * iper), ni = min(p.N - i0, iper);
  const int i = i0 + tid;
  const bool has_in = tid < nb, has_out = tid < ni;
  const int parent = has_out ? parent_of(p, i, err) : -1;
  const int have = has_in ? row_len(p, b0 + tid, err) : 0;
  const int scan_parent = tid < p.N ? p.parents[tid] : -1;
  Kin k{0, 0, 0};
  if (has_out) k = row_lengths(p, parent >= 0 ? row_len(p, parent, err) : 0, i, err);
  // the page the row's new keys begin in, where it holds keys
  const int at = parent >= 0 && k.want > k.keep && (k.keep & in_page) != 0 ? k.keep >> p.page_shift : -1;
  const int page = at >= 0 ? p.table[(size_t)parent * p.stride + at] : -1;
  const int last_page = (have & in_page) != 0 ? p.table[(size_t)(b0 + tid) * p.stride + (have >> p.page_shift)] : -1;
  s_kids[tid] = Kids{0, 0, INT_MAX, kSame};
  if (p.ref != p.ref_in)
    for (int x = (int)rank * kPlanThreads + tid; x < p.num_pages; x += kPlanCtas * kPlanThreads) p.ref[x] = p.ref_in[x];
  const bool alone = is_page(last_page, p.num_pages) && p.ref_in[last_page] == 1;
  __syncthreads();
  // a child that gives keys up adds kMaxCacheRows + 1 to g
  for (int x = tid; x < p.N; x += kPlanThreads) {
    const int b = (x == tid ? scan_parent : p.parents[x]) - b0;
    if (b < 0 || b >= nb) continue;
    uint32_t e = 0;
    const Kin c = row_lengths(p, row_len(p, b0 + b, e), x, e);
    atomicAdd(&s_kids[b].c, 1);
    if (c.want < c.have) atomicAdd(&s_kids[b].g, kMaxCacheRows + 1);
    if (c.want > c.have) {
      atomicAdd(&s_kids[b].g, 1);
      atomicMin(&s_kids[b].first, x);
    }
  }
  __syncthreads();
  if (has_in) {
    const int g = s_kids[tid].g;
    if (g > kMaxCacheRows) s_kids[tid].kind = kMixed;
    else if (g > 0 && (have & in_page) != 0 && !alone) s_kids[tid].kind = kClaims;
  }
  cluster_sync();
  auto kids_of = [&](int b) -> Kids {
    Kids c;
    const uint32_t from = map_to_rank(smem_addr(s_kids + b % bper), b / bper);
    asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(c.c), "=r"(c.g), "=r"(c.first), "=r"(c.kind)
                 : "r"(from)
                 : "memory");
    return c;
  };

  // 1: what this thread's output row does with the page its new keys begin in
  ForkRow r;
  r.src = parent;
  r.keep = k.keep;
  r.len = k.want;
  r.page = page;
  r.at = at;
  r.drop = drop_end(p, k.keep);
  bool claims = false, copy = false;
  if (at >= 0) {
    const Kids c = kids_of(parent);
    claims = c.kind != kSame;
    copy = claims || c.c != c.g || c.first != i;  // kSame: the first writer goes on if nobody only shares
  }
  // the counts: a warp an input row of this CTA, or an output row whose parent's children differ
  const int d0 = pages_of(p.sink_tokens, p.page_shift);
  constexpr int kU = 4, kChunk = 32 * kU;  // entries of an input row a warp takes at a time
  const int chunks = (p.stride + kChunk - 1) / kChunk;
  for (int item = warp; item < nb * chunks; item += kPlanThreads / 32) {
    const int b = item / chunks, base = item % chunks * kChunk;
    const Kids c = s_kids[b];
    uint32_t e0 = 0;
    const int keys = row_len(p, b0 + b, e0), n = pages_of(keys, p.page_shift);
    const bool mixed = c.kind == kMixed;
    const int d1 = mixed ? 0 : drop_end(p, keys);
    const int all = mixed ? -1 : c.c - 1;
    // the last page where rows write on: those that only share it, and (kSame) the one that has it if none does
    const int last = mixed ? -1 : c.c - c.g - 1 + (c.kind == kSame && c.c == c.g ? 1 : 0);
    const int lp = c.g > 0 && (keys & in_page) != 0 && last != all ? keys >> p.page_shift : -1;
    if (base >= n || (all == 0 && base >= d1 && lp < base)) continue;  // what changes: every page, or those given up and the last
    int e[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int j = base + 32 * u + lane;
      e[u] = j < n ? p.table[(size_t)(b0 + b) * p.stride + j] : MLA_NO_PAGE;
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int j = base + 32 * u + lane;
      if (j >= n) continue;
      const int d = c.c > 0 && !mixed && j >= d0 && j < d1 ? -1 : j == lp ? last : all;
      if (is_page(e[u], p.num_pages)) {
        if (d != 0) atomicAdd(p.ref + e[u], d);
      } else if (e[u] != MLA_NO_PAGE) {
        err |= kErrBadPage;
      }
    }
  }
  for (int x = i0 + warp; x < i0 + ni; x += kPlanThreads / 32) {
    const int b = p.parents[x];
    if (b < 0 || b >= p.B) continue;
    const bool mixed = kids_of(b).kind == kMixed, move = in_place && b != x;
    if (!mixed && !move) continue;
    uint32_t e0 = 0;
    const Kin c = row_lengths(p, row_len(p, b, e0), x, e0);
    const int n = pages_of(c.keep, p.page_shift), d1 = drop_end(p, c.keep);
    const int lp = c.want > c.keep && (c.keep & in_page) != 0 ? c.keep >> p.page_shift : -1;
    for (int j = lane; j < n; j += 32) {
      const int e = p.table[(size_t)b * p.stride + j];
      if (move) stage[(size_t)x * p.stride + j] = e;
      if (mixed && is_page(e, p.num_pages) && j != lp && !(j >= d0 && j < d1)) atomicAdd(p.ref + e, 1);
    }
  }
  bool any_claim = __syncthreads_or(claims);
  if (tid < kPlanCtas) st_shared_cluster(map_to_rank(smem_addr(&s_claims[rank]), tid), any_claim ? 1u : 0u);
  cluster_sync();

  // 2: claims
  any_claim = false;
  for (int c = 0; c < kPlanCtas; ++c) any_claim |= s_claims[c] != 0;
  if (any_claim) {
    const bool there = is_page(page, p.num_pages);
    if (claims && there && __ldcg(p.ref + page) <= 0) atomicMin(p.ref + page, claim_of(i));
    cluster_sync();
    if (claims && there) copy = __ldcg(p.ref + page) != claim_of(i);
    if (claims && !there) {
      err |= kErrBadPage;  // the page whose keys the row keeps is not there
      r.page = -1;
    }
  }

  // 3: needs and free pages (a warp's first 32 words stay in its lanes)
  const int need = (copy ? 1 : 0) + pages_of(r.len, p.page_shift) - pages_of(r.keep, p.page_shift);
  int w0, w1;
  my_words(p.num_pages, rank, warp, w0, w1);
  uint32_t mine;
  int fbase = scan_words(p.ref, p.num_pages, w0, w1, words, mine, [](int v) { return v <= 0 && !is_claim(v); });
  int off = __reduce_add_sync(0xffffffffu, need), cta_need, cta_free;
  const int before_me = off > 0 ? lane_prefix(need) : 0;
  warp_sums(off, part[0], cta_need);
  warp_sums(fbase, part[1], cta_free);
  off += before_me;
  publish(s_sums, rank, cta_need, cta_free);
  cluster_sync();

  // 4: places
  int2 before, all;
  collect(s_sums, rank, before, all);
  off += before.x;
  fbase += before.y;
  const int avail = all.y, most = min(all.x, avail);
  if (has_out) {
    if (claims && !copy) p.ref[page] = 1;
    r.fresh = off;
    r.nfresh = need;
    if (need > 0 && off + need > avail) {
      err |= kErrNoPages;
      r.nfresh = 0;
      r.len = copy ? r.keep & ~in_page : r.keep;
      if (copy) r.keep = r.len;
      copy = false;
    }
    if (!copy) r.at = -1;
    reinterpret_cast<int4*>(info + i)[0] = reinterpret_cast<const int4*>(&r)[0];
    reinterpret_cast<int4*>(info + i)[1] = reinterpret_cast<const int4*>(&r)[1];
  }
  for (int w = w0; w < w1 && fbase < most; ++w) {
    const uint32_t m = word_of(words, mine, w0, w);
    const int f = fbase + __popc(m & ((1u << lane) - 1u));
    if ((m >> lane & 1u) != 0 && f < most) list[f] = 32 * w + lane;
    fbase += __popc(m);
  }
  flag(p.status, err);
}

// The rows as planned: a block a row (and slice: the four slices share the copy of the page the
// row writes on in).  Launched with the plan, it waits for it on the other SMs.
__global__ void __launch_bounds__(256) fork_rows_kernel(const __grid_constant__ ForkParams p) {
  grid_dependency_wait();
  const CacheWs L = cache_ws(p.num_pages, p.stride, p.ws_rows);
  const int i = blockIdx.x;
  const ForkRow r = reinterpret_cast<const ForkRow*>(p.ws + L.rows)[i];
  const int32_t* list = reinterpret_cast<const int32_t*>(p.ws + L.list) + r.fresh;
  const bool copies = r.at >= 0;
  if (blockIdx.y == 0) {
    const bool staged = p.table == p.table_out && r.src != i;
    const int32_t* row = staged ? reinterpret_cast<const int32_t*>(p.ws + L.stage) + (size_t)i * p.stride
                                : p.table + (size_t)max(r.src, 0) * p.stride;
    int32_t* out = p.table_out + (size_t)i * p.stride;
    const int pk = pages_of(r.keep, p.page_shift), pn = r.nfresh > 0 ? pages_of(r.len, p.page_shift) : pk;
    const int d0 = pages_of(p.sink_tokens, p.page_shift), d1 = r.drop;
    for (int j = threadIdx.x; j < p.stride; j += blockDim.x) {
      int e = MLA_NO_PAGE;
      bool fresh = false;
      if (copies && j == r.at) {
        e = list[0];
        fresh = true;
      } else if (j < pk) {
        if (!(j >= d0 && j < d1)) {
          e = row[j];
          if (!is_page(e, p.num_pages)) e = MLA_NO_PAGE;
        }
      } else if (j < pn) {
        e = list[(copies ? 1 : 0) + j - pk];
        fresh = true;
      }
      out[j] = e;
      if (fresh) p.ref[e] = 1;
    }
    if (threadIdx.x == 0) {
      p.lens_out[i] = r.len;
      if (p.kept) p.kept[i] = r.keep;
    }
  }
  if (copies && r.page >= 0) {
    const int slots = r.keep & ((1 << p.page_shift) - 1);
    const int units = slots * (kDQK * p.es / 16);
    const int per = ((units + gridDim.y - 1) / gridDim.y + 31) & ~31;
    const int u0 = min(units, (int)blockIdx.y * per);
    copy_slots(p.ckv, p.kpe, p.ckv, p.kpe, r.page, list[0], p.page_shift, p.es, u0, min(units, u0 + per), slots,
               threadIdx.x, blockDim.x);
  }
}

// ------------------------------------------------------------------ compact
// One cluster: the pages in use (n of them) are counted; the m-th of those at n or above goes
// to the m-th free page below n.  Phases as in the fork, a cluster barrier between them.
// Measured with the moves: 500 pages 7.2 us, a pool of 16384 64-key bf16 pages half in use
// (4096 of them moved, 605 MB) 97.0 us (6.2 TB/s).
__global__ void __launch_bounds__(kPlanThreads, 1) compact_plan_kernel(const __grid_constant__ CompactParams p) {
  __shared__ int part[32], s_below;
  __shared__ int2 s_sums[kPlanCtas];
  const uint32_t rank = cluster_ctarank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const CacheWs L = cache_ws(p.num_pages, p.stride, p.ws_rows);
  int32_t* counts = reinterpret_cast<int32_t*>(p.ws + L.counts);
  uint32_t* words = reinterpret_cast<uint32_t*>(p.ws + L.words);
  const int half = p.num_pages / 2 + 1;
  int32_t* holes = reinterpret_cast<int32_t*>(p.ws + L.list);
  int32_t* moved = holes + half;
  int32_t* moved_ref = moved + half;
  grid_launch_dependents();
  cluster_arrive();  // this CTA runs: its shared memory may be written from the others
  int w0, w1;
  my_words(p.num_pages, rank, warp, w0, w1);
  uint32_t mine;
  int base = scan_words(p.ref_in, p.num_pages, w0, w1, words, mine, [](int v) { return v > 0; });
  int cta_used;
  warp_sums(base, part, cta_used);
  cluster_wait();
  publish(s_sums, rank, cta_used, 0);
  cluster_sync();
  int2 before, sums;
  collect(s_sums, rank, before, sums);
  base += before.x;
  const int n = sums.x;
  // used pages below n: of the word that holds page n, the part before it
  {
    int run = base, below = -1;
    for (int w = w0; w < w1; ++w) {
      const uint32_t m = word_of(words, mine, w0, w);
      if (n >= 32 * w && n < 32 * w + 32) below = run + __popc(m & ((1u << (n & 31)) - 1u));
      run += __popc(m);
    }
    // n at the end of the pool: every page is in use
    if (rank == 0 && warp == 0 && n >= ((p.num_pages + 31) / 32) * 32) below = n;
    if (lane < kPlanCtas && below >= 0) st_shared_cluster(map_to_rank(smem_addr(&s_below), lane), (uint32_t)below);
  }
  cluster_sync();
  const int below = s_below;
  {
    int run = base;
    for (int w = w0; w < w1; ++w) {
      const uint32_t m = word_of(words, mine, w0, w);
      const int x = 32 * w + lane;
      const int rk = run + __popc(m & ((1u << lane) - 1u));  // used pages before x
      run += __popc(m);
      if (x >= p.num_pages) continue;
      const bool used = (m >> lane) & 1u;
      if (used && x >= n) {
        moved[rk - below] = x;
        moved_ref[rk - below] = p.ref_in[x];
      } else if (!used && x < n) {
        holes[x - rk] = x;
      }
    }
  }
  if (rank == 0 && tid == 0) {
    counts[0] = n - below;
    *p.num_used = n;
  }
  cluster_sync();
  {
    int run = base;
    for (int w = w0; w < w1; ++w) {
      const uint32_t m = word_of(words, mine, w0, w);
      const int x = 32 * w + lane;
      const int rk = run + __popc(m & ((1u << lane) - 1u));
      run += __popc(m);
      if (x >= p.num_pages) continue;
      const bool used = (m >> lane) & 1u;
      int to = MLA_NO_PAGE, ref = 0;
      if (used && x < n) {
        to = x;
        ref = p.ref_in[x];
      } else if (used) {
        to = __ldcg(holes + (rk - below));
      } else if (x < n) {
        ref = __ldcg(moved_ref + (x - rk));
      }
      p.page_map[x] = to;
      p.ref[x] = ref;
    }
  }
}

__global__ void __launch_bounds__(kCopyThreads) compact_move_kernel(const __grid_constant__ CompactParams p) {
  grid_dependency_wait();
  const CacheWs L = cache_ws(p.num_pages, p.stride, p.ws_rows);
  const size_t n = (size_t)p.B * p.stride;
  for (size_t x = (size_t)blockIdx.x * blockDim.x + threadIdx.x; x < n; x += (size_t)gridDim.x * blockDim.x) {
    const int e = p.table[x];
    p.table_out[x] = is_page(e, p.num_pages) ? p.page_map[e] : e;
  }
  const int half = p.num_pages / 2 + 1;
  const int32_t* holes = reinterpret_cast<const int32_t*>(p.ws + L.list);
  const int moves = reinterpret_cast<const int32_t*>(p.ws + L.counts)[0];
  copy_pages(p.ckv, p.kpe, p.ckv, p.kpe, holes + half, holes, moves, p.num_pages, p.num_pages, p.page_shift, p.es, nullptr);
}

// What a launch needs of the current device, found on its first call there (a cluster of 16 has
// to be allowed once per kernel): asking again costs the host a microsecond a call.
struct DeviceInfo {
  int sms;
  cudaError_t error;
};
DeviceInfo device_info() {
  static std::atomic<int> known[64];
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return {0, e};
  const bool keep = dev >= 0 && dev < 64;
  if (keep && (sms = known[dev].load(std::memory_order_acquire)) > 0) return {sms, cudaSuccess};
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) == cudaSuccess &&
      (e = cudaFuncSetAttribute(fork_plan_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) == cudaSuccess &&
      (e = cudaFuncSetAttribute(compact_plan_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) == cudaSuccess && keep)
    known[dev].store(sms, std::memory_order_release);
  return {sms, e};
}

// one cluster of kPlanCtas
template <typename P>
cudaError_t launch_plan(void (*kernel)(P), const P& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kPlanCtas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = kPlanCtas;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <typename P>
cudaError_t launch_dependent(void (*kernel)(P), const P& p, dim3 grid, int threads, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_append(const AppendParams& p, bool in_f32, bool e4m3, cudaStream_t stream) {
  const DeviceInfo d = device_info();
  if (d.error != cudaSuccess) return d.error;
  const int all = (p.num_tokens + kAppendWarps - 1) / kAppendWarps;
  const int blocks = all < d.sms * kAppendWave ? all : d.sms * kAppendWave;
  if (in_f32) {
    if (e4m3) append_kernel<float, true><<<blocks, kAppendThreads, 0, stream>>>(p);
    else append_kernel<float, false><<<blocks, kAppendThreads, 0, stream>>>(p);
  } else {
    if (e4m3) append_kernel<__nv_bfloat16, true><<<blocks, kAppendThreads, 0, stream>>>(p);
    else append_kernel<__nv_bfloat16, false><<<blocks, kAppendThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

cudaError_t launch_fork(const ForkParams& p, cudaStream_t stream) {
  const DeviceInfo d = device_info();
  if (d.error != cudaSuccess) return d.error;
  cudaError_t e = launch_plan(fork_plan_kernel, p, stream);
  if (e != cudaSuccess || p.N == 0) return e;
  return launch_dependent(fork_rows_kernel, p, dim3((unsigned)p.N, 4), 256, stream);
}

cudaError_t launch_compact(const CompactParams& p, cudaStream_t stream) {
  const DeviceInfo d = device_info();
  if (d.error != cudaSuccess) return d.error;
  cudaError_t e = launch_plan(compact_plan_kernel, p, stream);
  if (e != cudaSuccess) return e;
  return launch_dependent(compact_move_kernel, p, dim3((unsigned)(d.sms * kMoveWave)), kCopyThreads, stream);
}

cudaError_t launch_copy(const CopyParams& p, cudaStream_t stream) {
  const DeviceInfo d = device_info();
  if (d.error != cudaSuccess) return d.error;
  const long long blocks = (((long long)p.n << runs_shift(p.page_shift, p.es)) + kCopyWarps - 1) / kCopyWarps;
  const long long most = (long long)d.sms * kCopyWave;
  copy_kernel<<<(unsigned)(blocks < most ? blocks : most), kCopyThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace mla
