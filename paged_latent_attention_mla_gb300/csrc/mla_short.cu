// Decode of short spans: few (token, head) rows over few visible keys, where the split-KV
// kernel's fixed cost is the call.
//
// One cluster per tile of 16, 32 or 64 rows of a request (short_shape chooses): its C CTAs take equal runs of the
// tile's 64-key groups (the sinks' groups, then the window's), each runs the one-pass softmax
// over its own, and the cluster joins the parts through distributed shared memory: one launch,
// no workspace traffic, no second kernel.  A group is loaded once (its latents are K and V both):
// nine [64 keys x 128 B] blocks by TMA, two groups in flight, read by ldmatrix through the
// 128-byte swizzle, straight for Q.K^T and transposed for P.V.  The products are warp-level
// 16-bit MMAs: a group of one row tile has 8.9 MFLOP at most, and a kernel that small in code
// starts in 3 us where the tensor-memory kernel's roles, schedule and teardown take 20.
//
// Measured (GB300, back to back): one request of 16 heads over 256, 1024 and 4096 keys 8.9, 9.5
// and 15.3 us (split-KV kernel and reduction 18.2, 21.8, 26.3).  A CTA takes 7 us besides its
// groups (launch 1, lengths 0.6, page ids 1.3, first copies 0.6, join 3.5) and per group 2.0 us at 16 rows,
// 2.7 at 32 and 4.5 at 64: at 64 its 544 MMAs per scheduler, 16 cycles each, are that time; at
// 16 they are half of it, the rest the waits between the steps below.  With an e4m3 cache the
// three take 10.4, 11.1 and 18.9 us (16.4, 19.6, 24.0), 2.7 us per group.
//
// An e4m3 cache's groups land as they are (two in flight, 36 KB each) and are widened to fp16, exactly,
// into one stage the products read; Q likewise, once.  P is then fp16 (each p off by 2^-11 of itself,
// 2^-25 at the smallest), so the result is closer than with the split-KV kernel's e4m3 P.
//
// Per group: S = Q.K^T (warp: 16 rows x 64 / warps-per-row-tile keys), row maxima meet in shared
// memory, P = 2^(S - m) to shared memory as bf16 (each p off by 2^-8 of itself, as in the
// split-KV kernel; the row sums add the unrounded p in fp32), O += P.c (warp: 64 of the 512
// dims, all rows; fp32 in registers).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "mla_common.cuh"
#include "mla_kernels.cuh"
#include "ptx.cuh"
#include "schedule.cuh"
#include "tma_pages.cuh"

namespace mla {
namespace {

constexpr int kShortThreads = 256, kShortWarps = kShortThreads / 32;
constexpr int kBlocks = kDQK / 64;                // column blocks of a key: 8 latent, 1 rope
constexpr int kStageBytes = kBlocks * kBlockBytes;  // one 64-key group, or the Q tile
struct ShortMisc {
  uint64_t full[2], q_full;
  float row_max[kShortWarps][16];  // [warp of the row tile][row], RT tiles of 16 rows side by side
  float row_sum[kShortWarps][16];
  float fac[64];
  float m[64], l[64];              // the CTA's rows, read by the cluster
  uint32_t ok, err;
};
constexpr int kRawBytes = 4 * kBlockBytes + 64 * 64;  // an e4m3 group, or Q tile, as it lands
constexpr int kOffK = kStageBytes, kOffRaw = 2 * kStageBytes, kOffP = 3 * kStageBytes, kOffMisc = kOffP + kBlockBytes;
constexpr int kShortSmem = kOffMisc + (int)sizeof(ShortMisc) + 1024;
static_assert(kShortSmem <= 232448, "exceeds shared memory");
static_assert(kOffRaw + 2 * kRawBytes <= kOffP && kRawBytes % 1024 == 0, "the landing buffers");
constexpr int kOStride = kDLatent + 8;  // floats between rows of O in shared memory: no bank conflicts
static_assert(64 * kOStride * 4 <= 2 * kStageBytes, "O over the two stages");

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <bool F16>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  if constexpr (F16) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// 16 e4m3 values at `from` to 16 fp16 values, chunks c and c + 1 of a swizzled row
__device__ __forceinline__ void widen16(const uint8_t* from, uint8_t* to_row, int c, int row, bool keep) {
  const uint4 v = keep ? *reinterpret_cast<const uint4*>(from) : make_uint4(0, 0, 0, 0);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t h[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[e / 2] >> (16 * (e & 1))), __NV_E4M3);
    h[e] = static_cast<uint32_t>(r.x) | static_cast<uint32_t>(r.y) << 16;
  }
  *reinterpret_cast<uint4*>(to_row + ((c ^ (row & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
  *reinterpret_cast<uint4*>(to_row + (((c + 1) ^ (row & 7)) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
}
// 64 rows of e4m3 as they landed (four [64 x 128 B] blocks, 128-byte swizzle, and the rope's
// [64 x 64 B], 64-byte swizzle) to nine fp16 blocks, rows from `valid` on as zeros (their bits
// may be anything).  All threads of the block.  Eight lanes of a latent block take four chunks of
// the rows r and r ^ 5: the reads then differ in the swizzle's bit 2 and the writes, whose chunks
// go by twos, in its bit 0, so neither meets on a bank.
template <int kUnroll>
__device__ __forceinline__ void widen(const uint8_t* raw, uint8_t* dst, int valid, int tid) {
  static_assert(kShortThreads == 256, "two rounds to a latent block, one to the rope's");
#pragma unroll kUnroll
  for (int t = 0; t < 8; ++t) {
    const int y = (t & 1) * 256 + tid;
    const int row = (((y >> 3) & 3) ^ (((y >> 2) & 1) * 5)) | (y >> 6) << 3, ch = (y & 3) | ((y >> 5) & 1) << 2;
    widen16(raw + (t >> 1) * kBlockBytes + row * 128 + ((ch ^ (row & 7)) << 4),
            dst + ((t >> 1) * 2 + (ch >> 2)) * kBlockBytes + row * 128, 2 * (ch & 3), row, row < valid);
  }
  const int row = tid >> 2, ch = tid & 3;
  widen16(raw + 4 * kBlockBytes + row * 64 + ((ch ^ ((row >> 1) & 3)) << 4), dst + 8 * kBlockBytes + row * 128, 2 * ch, row,
          row < valid);
}
// 2^x with the hardware approximation (relative error ~2^-22; denormal results flush to 0)
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

// RT: tiles of 16 rows to a CTA (1, 2 or 4); E4M3: an e4m3 cache and queries (else bf16)
template <int RT, bool E4M3>
__global__ void __launch_bounds__(kShortThreads, 1) short_decode(const __grid_constant__ DecodeParams p,
                                                                 const __grid_constant__ KvMaps maps) {
  constexpr int kRows = 16 * RT;
  constexpr int kPer = kShortWarps / RT;  // warps of a row tile, a share of the group's keys each
  constexpr int kCols = blk_elems<E4M3>(), kLat = latent_blocks<E4M3>(), kRopeRow = E4M3 ? 64 : 128;  // as loaded
  constexpr uint32_t kLanded = E4M3 ? kRawBytes : kStageBytes;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  ShortMisc& M = *reinterpret_cast<ShortMisc*>(smem + kOffMisc);
  const uint32_t sQ = smem_addr(smem), sK = sQ + kOffK, sP = sQ + kOffP;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x, C = gridDim.x;
  const int rows_q = p.Sq * p.H, tiles = (rows_q + kRows - 1) / kRows;
  const int b = blockIdx.y / tiles, flat0 = blockIdx.y % tiles * kRows;

  if (tid == 0) {
    M.err = 0;
    mbar_init(smem_addr(&M.full[0]), 1);
    mbar_init(smem_addr(&M.full[1]), 1);
    mbar_init(smem_addr(&M.q_full), 1);
    fence_mbar_init();
  }
  __syncthreads();
  // this CTA's run of the tile's groups
  const int K = clamp_len(p, b, rank == 0 && tid == 0 ? &M.err : nullptr), Kg = global_len(p, b, K);
  const KeySpan span = window_span<kSinks>(tokens_span(p, b, flat0 / p.H, (min(rows_q, flat0 + kRows) - 1) / p.H, K, Kg), K);
  const Groups g = key_groups(span, p.sinks);
  const int Kv = span.end;
  const int per = (g.n + C - 1) / C;
  const int v0 = min(g.n, rank * per), v1 = min(g.n, v0 + per), n = v1 - v0;
  const int parts = per > 0 ? (g.n + per - 1) / per : 0;  // CTAs of the cluster with groups

  // warp 0 loads: lane q the page of box q of a group, a group ahead of its copies (a round trip
  // that would otherwise be part of every copy's), then a box a lane
  const int br = box_rows(p.page_size), nbs = max(0, 6 - p.page_shift), nb = 1 << nbs;  // boxes of br keys to a group
  int pg = p.num_pages, rw = 0;
  bool bad = false;
  auto look_up = [&](int i) {
    if (i >= n || lane >= nb) return;
    bool miss;
    box_page<kSinks>(p.page_table, p.pt_stride, p.num_pages, p.page_shift, b, g.at(v0 + i) * kKeyGroup + lane * br, br,
                   span.lo, p.sinks, Kv, pg, rw, miss);
    bad |= miss;
  };
  auto load = [&](int i) {
    const uint32_t bar = smem_addr(&M.full[i & 1]);
    const uint32_t dst = E4M3 ? sQ + kOffRaw + (i & 1) * kRawBytes : sK + (i & 1) * kStageBytes;
    if (lane == 0) mbar_arrive_expect_tx(bar, kLanded);
    __syncwarp();
    for (int x0 = 0; x0 < (kLat + 1) * nb; x0 += 32) {
      const int x = x0 + lane, kb = x >> nbs, q = x & (nb - 1);
      const int page = __shfl_sync(0xffffffffu, pg, q), row = __shfl_sync(0xffffffffu, rw, q);
      if (x >= (kLat + 1) * nb) continue;
      const uint32_t d = dst + kb * kBlockBytes + q * br * (kb < kLat ? 128 : kRopeRow);
      if (kb < kLat) tma_load_3d(d, &maps.ckv, kb * kCols, row, page, bar);
      else tma_load_3d(d, &maps.kpe, 0, row, page, bar);
    }
    look_up(i + 1);
  };
  if (warp == 0 && n > 0) {
    look_up(0);
    if (lane == 0) mbar_arrive_expect_tx(smem_addr(&M.q_full), kLanded);
    __syncwarp();
    const uint32_t q_at = E4M3 ? sK : sQ;  // e4m3: on the stage, until it is widened
    if (lane < kLat) tma_load_3d(q_at + lane * kBlockBytes, &maps.q_latent, lane * kCols, flat0, b, smem_addr(&M.q_full));
    else if (lane == kLat) tma_load_3d(q_at + kLat * kBlockBytes, &maps.q_rope, 0, flat0, b, smem_addr(&M.q_full));
    load(0);
    if (n > 1) load(1);
  }

  // this thread's two rows of S: their tokens' keys
  const int rt = warp % RT, part = warp / RT;
  const int row0 = 16 * rt + (lane >> 2);
  int lo[2] = {0, 0}, hi[2] = {0, 0};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int flat = flat0 + row0 + 8 * h;
    if (flat < rows_q) token_keys(p, b, flat / p.H, K, Kg, lo[h], hi[h]);
  }
  const float cl2 = p.score_scale_log2;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  float o[RT][8][4];
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[t][j][e] = 0.f;

  uint32_t qf[RT == 1 ? 4 * kBlocks : 1][4];
  for (int i = 0; i < n; ++i) {
    const uint32_t bar = smem_addr(&M.full[i & 1]), stage = E4M3 ? sK : sK + (i & 1) * kStageBytes;
    // one thread's bounded wait decides for all; the others then see the phase complete
    if (tid == 0)
      M.ok = (i > 0 || mbar_wait_bounded(smem_addr(&M.q_full), 0, kWaitTimeoutNs)) &&
             mbar_wait_bounded(bar, (i >> 1) & 1, kWaitTimeoutNs);
    __syncthreads();
    if (!M.ok) {
      if (tid == 0) {
        atomicOr(&M.err, kErrTimeout);
        // the copies still in flight land in this CTA's memory: give them one more time limit
        mbar_wait_bounded(smem_addr(&M.q_full), 0, kWaitTimeoutNs);
        for (int x = i; x < min(n, E4M3 || i == 0 ? i + 2 : i + 1); ++x)
          mbar_wait_bounded(smem_addr(&M.full[x & 1]), (x >> 1) & 1, kWaitTimeoutNs);
      }
      break;
    }
    if (i == 0) mbar_try_wait(smem_addr(&M.q_full), 0);
    mbar_try_wait(bar, (i >> 1) & 1);
    const int key0 = g.at(v0 + i) * kKeyGroup;
    // slots past the keys that are read: any bits there must not reach P.c
    if constexpr (E4M3) {
      if (i == 0) {
        widen<1>(smem + kOffK, smem, 64, tid);
        __syncthreads();
      }
      widen<RT == 4 ? 2 : 4>(smem + kOffRaw + (i & 1) * kRawBytes, smem + kOffK, Kv - key0, tid);  // RT 4: 4 spills
      __syncthreads();
      // the group as it landed is read: the one after next goes there
      if (warp == 0 && i + 2 < n) load(i + 2);
    } else {
      // every warp is done with the other stage: the next group goes there
      if (warp == 0 && i > 0 && i + 1 < n) load(i + 1);
      if (key0 + kKeyGroup > Kv) {
        for (int kb = 0; kb < 8; ++kb)
          zero_block_rows(smem + kOffK + (i & 1) * kStageBytes + kb * kBlockBytes, max(Kv - key0, 0), tid, kShortThreads);
        fence_proxy_async_smem();
        __syncthreads();
      }
    }

    // S: rows 16 rt .., keys 8 RT part ..  At least four sums run side by side (an MMA waits for
    // the one before it on the same sum): kSplit of the 16-dim steps' sums to a tile of keys.
    constexpr int kSplit = 4 / RT;
    float s[RT][4], sp[RT][kSplit][4];
#pragma unroll
    for (int j = 0; j < RT; ++j)
#pragma unroll
      for (int q = 0; q < kSplit; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) sp[j][q][e] = 0.f;
    const int arow = 16 * rt + (lane & 15);
    if constexpr (RT == 1) {
      // every warp needs all of Q: from registers, else its reads are most of the group's
      if (i == 0) {
#pragma unroll
        for (int kk = 0; kk < 4 * kBlocks; ++kk)
          ldsm4(sQ + kk / 4 * kBlockBytes + arow * 128 + (((2 * (kk % 4) + (lane >> 4)) ^ (arow & 7)) << 4), qf[kk]);
      }
      // one n-tile: the B operands of two 16-dim steps to a load
      const int krow = 8 * part + (lane & 7);
#pragma unroll
      for (int kk = 0; kk < 4 * kBlocks; kk += 2) {
        uint32_t bf[4];
        ldsm4(stage + kk / 4 * kBlockBytes + krow * 128 + (((2 * (kk % 4) + (lane >> 3)) ^ (krow & 7)) << 4), bf);
        mma16<E4M3>(sp[0][kk % 4], qf[kk], bf[0], bf[1]);
        mma16<E4M3>(sp[0][kk % 4 + 1], qf[kk + 1], bf[2], bf[3]);
      }
    } else {
#pragma unroll 3
      for (int kb = 0; kb < kBlocks; ++kb) {
        const uint32_t qa = sQ + kb * kBlockBytes + arow * 128, ka = stage + kb * kBlockBytes;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          uint32_t a[4];
          ldsm4(qa + (((2 * ks + (lane >> 4)) ^ (arow & 7)) << 4), a);
#pragma unroll
          for (int j = 0; j < RT; j += 2) {
            const int krow = 8 * (RT * part + j + (lane >> 4)) + (lane & 7);
            uint32_t bf[4];
            ldsm4(ka + krow * 128 + (((2 * ks + ((lane >> 3) & 1)) ^ (krow & 7)) << 4), bf);
            mma16<E4M3>(sp[j][ks % kSplit], a, bf[0], bf[1]);
            mma16<E4M3>(sp[j + 1][ks % kSplit], a, bf[2], bf[3]);
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < RT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[j][e] = sp[j][0][e];
#pragma unroll
        for (int q = 1; q < kSplit; ++q) s[j][e] += sp[j][q][e];
      }
    // mask, row maxima over the tile's warps
    float mt[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int j = 0; j < RT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int h = e >> 1, key = key0 + 8 * (RT * part + j) + 2 * (lane & 3) + (e & 1);
        const bool vis = key < hi[h] && (key >= lo[h] || key < p.sinks);
        s[j][e] = vis ? s[j][e] * cl2 : -INFINITY;
        mt[h] = fmaxf(mt[h], s[j][e]);
      }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      mt[h] = fmaxf(mt[h], __shfl_xor_sync(0xffffffffu, mt[h], 1));
      mt[h] = fmaxf(mt[h], __shfl_xor_sync(0xffffffffu, mt[h], 2));
      if ((lane & 3) == 0) M.row_max[part * RT + rt][(lane >> 2) + 8 * h] = mt[h];
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float mn = m[h];
#pragma unroll
      for (int q = 0; q < kPer; ++q) mn = fmaxf(mn, M.row_max[q * RT + rt][(lane >> 2) + 8 * h]);
      // no key seen so far: every p is 2^-inf, whatever the reference
      const float fac = mn == -INFINITY ? 1.f : exp2_fast(m[h] - mn);
      m[h] = mn;
      l[h] *= fac;
      const float ref = mn == -INFINITY ? 0.f : mn;
      const int row = row0 + 8 * h;
      if (part == 0 && (lane & 3) == 0) M.fac[row] = fac;
#pragma unroll
      for (int j = 0; j < RT; ++j) {
        const float p0 = exp2_fast(s[j][2 * h] - ref), p1 = exp2_fast(s[j][2 * h + 1] - ref);
        l[h] += p0 + p1;
        const int chunk = RT * part + j;
        *reinterpret_cast<uint32_t*>(smem + kOffP + row * 128 + ((chunk ^ (row & 7)) << 4) + 4 * (lane & 3)) =
            pack2<E4M3>(p0, p1);
      }
    }
    __syncthreads();
    // O = O fac + P.c, dims 64 warp ..
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const float f0 = M.fac[16 * t + (lane >> 2)], f1 = M.fac[16 * t + (lane >> 2) + 8];
      if (__any_sync(0xffffffffu, f0 != 1.f || f1 != 1.f)) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          o[t][j][0] *= f0;
          o[t][j][1] *= f0;
          o[t][j][2] *= f1;
          o[t][j][3] *= f1;
        }
      }
    }
    const uint32_t va = stage + warp * kBlockBytes;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      uint32_t a[RT][4];
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        const int prow = 16 * t + (lane & 15);
        ldsm4(sP + prow * 128 + (((2 * ks + (lane >> 4)) ^ (prow & 7)) << 4), a[t]);
      }
      const int vrow = 16 * ks + (lane & 15);
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        uint32_t bf[4];
        ldsm4_trans(va + vrow * 128 + (((j + (lane >> 4)) ^ (vrow & 7)) << 4), bf);
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          mma16<E4M3>(o[t][j], a[t], bf[0], bf[1]);
          mma16<E4M3>(o[t][j + 1], a[t], bf[2], bf[3]);
        }
      }
    }
  }
  if (bad) atomicOr(&M.err, kErrBadPage);
  __syncthreads();  // the last group's reads are done: O goes over the stages

  // the CTA's part: O (not normalized), row maxima and sums
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    if ((lane & 3) == 0) {
      M.row_sum[part * RT + rt][(lane >> 2) + 8 * h] = l[h];
      if (part == 0) M.m[row0 + 8 * h] = m[h];
    }
  }
  float* so = reinterpret_cast<float*>(smem + kOffK);
  if (n > 0) {
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<float2*>(so + (16 * t + (lane >> 2) + 8 * h) * kOStride + 64 * warp + 8 * j + 2 * (lane & 3)) =
              make_float2(o[t][j][2 * h], o[t][j][2 * h + 1]);
  }
  __syncthreads();
  if (tid < kRows) {
    float sum = 0.f;
#pragma unroll
    for (int q = 0; q < kPer; ++q) sum += M.row_sum[q * RT + tid / 16][tid % 16];
    M.l[tid] = sum;
  }
  cluster_sync();

  // join: this CTA the dims [rank D, rank D + D) of every row.  Weights 2^(m_c - m) / sum of the
  // parts into the P buffer, [part][row]: a lane a part, 16 lanes a row.
  float* sw = reinterpret_cast<float*>(smem + kOffP);
  static_assert(kMaxShortCtas == 16 && kMaxShortCtas * kRows * 4 <= kBlockBytes, "the parts' weights over P");
  for (int x = tid; x < kMaxShortCtas * kRows; x += kShortThreads) {
    const int row = x >> 4, c = x & 15;
    float mc = -INFINITY, lc = 0.f;
    if (c < parts) {
      mc = __uint_as_float(ld_shared_cluster(map_to_rank(smem_addr(M.m + row), c)));
      lc = __uint_as_float(ld_shared_cluster(map_to_rank(smem_addr(M.l + row), c)));
    }
    float mx = mc;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float w = exp2f(mc - (mx == -INFINITY ? 0.f : mx));
    float sum = w * lc;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    sw[c * kRows + row] = sum > 0.f ? w * (p.ckv_descale / sum) : 0.f;
    if (c == 0 && rank == 0 && p.lse && flat0 + row < rows_q)
      p.lse[(size_t)b * rows_q + flat0 + row] = sum > 0.f ? (mx + log2f(sum)) * 0.69314718055994530942f : -INFINITY;
  }
  __syncthreads();
  const int D = kDLatent / C, quads = D / 4, turn = parts > 0 ? rank % parts : 0;
  for (int x = tid; x < kRows * quads; x += kShortThreads) {
    const int row = x / quads, d = rank * D + x % quads * 4;
    if (flat0 + row >= rows_q) break;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const uint32_t at = smem_addr(so + row * kOStride + d);
    if (parts == 1) {
      const float w = sw[row];
      const float4 v = ld_cluster4(map_to_rank(at, 0));
      acc = make_float4(w * v.x, w * v.y, w * v.z, w * v.w);
    }
    // kU parts read at a time (a remote read takes 0.2 us), each CTA beginning with another one
    constexpr int kU = 16 / RT;
    for (int c0 = 0; c0 < parts && parts > 1; c0 += kU) {
      float4 v[kU];
      float w[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        int c = c0 + u + turn;
        if (c >= parts) c -= parts;
        w[u] = 0.f;
        v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c0 + u < parts) {
          v[u] = ld_cluster4(map_to_rank(at, c));
          w[u] = sw[c * kRows + row];
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        acc.x += w[u] * v[u].x;
        acc.y += w[u] * v[u].y;
        acc.z += w[u] * v[u].z;
        acc.w += w[u] * v[u].w;
      }
    }
    const size_t to = ((size_t)b * rows_q + flat0 + row) * kDLatent + d;
    if (p.out_f32) {
      *reinterpret_cast<float4*>(static_cast<float*>(p.out) + to) = acc;
    } else {
      const __nv_bfloat162 a = __floats2bfloat162_rn(acc.x, acc.y), c = __floats2bfloat162_rn(acc.z, acc.w);
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + to) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&c));
    }
  }
  // the status the workspace keeps, as the split-KV kernel leaves it
  if (tid == 0) {
    uint32_t* words = reinterpret_cast<uint32_t*>(p.ws + align256(sizeof(WsHeader)));
    const int ctas = gridDim.x * gridDim.y, me = blockIdx.y * gridDim.x + blockIdx.x;
    words[me] = M.err;
    if (me == 0) {
      if (ctas & 1) words[ctas] = 0;
      WsHeader* hd = reinterpret_cast<WsHeader*>(p.ws);
      *hd = WsHeader{0, (int)gridDim.y, (ctas + 1) / 2, 0, 0, 0, 0, 0};
    }
  }
  cluster_sync();  // the others may still read this CTA's memory
}

template <int RT, bool E4M3>
cudaError_t launch_short_variant(const DecodeParams& p, const KvMaps& maps, int C, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)C, (unsigned)(p.B * cdiv(p.Sq * p.H, 16 * RT)));
  cfg.blockDim = dim3(kShortThreads);
  cfg.dynamicSmemBytes = kShortSmem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)C;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, short_decode<RT, E4M3>, p, maps);
}

template <int RT, bool E4M3>
int max_clusters(int C) {
  if (cudaFuncSetAttribute(short_decode<RT, E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, kShortSmem) != cudaSuccess ||
      cudaFuncSetAttribute(short_decode<RT, E4M3>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
    cudaGetLastError();  // the next launch's check is not to find this error
    return 0;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)C, 64);
  cfg.blockDim = dim3(kShortThreads);
  cfg.dynamicSmemBytes = kShortSmem;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)C;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, short_decode<RT, E4M3>, &cfg) == cudaSuccess) return n;
  cudaGetLastError();
  return 0;
}

}  // namespace

int short_max_clusters(ShortShape s, bool e4m3) {
  if (s.rows == 16) return e4m3 ? max_clusters<1, true>(s.ctas) : max_clusters<1, false>(s.ctas);
  if (s.rows == 32) return e4m3 ? max_clusters<2, true>(s.ctas) : max_clusters<2, false>(s.ctas);
  return e4m3 ? max_clusters<4, true>(s.ctas) : max_clusters<4, false>(s.ctas);
}

cudaError_t launch_short(const DecodeParams& p, const KvMaps& maps, ShortShape s, cudaStream_t stream) {
  const int C = s.ctas;
  if (p.qkv_e4m3) {
    if (s.rows == 16) return launch_short_variant<1, true>(p, maps, C, stream);
    if (s.rows == 32) return launch_short_variant<2, true>(p, maps, C, stream);
    return launch_short_variant<4, true>(p, maps, C, stream);
  }
  if (s.rows == 16) return launch_short_variant<1, false>(p, maps, C, stream);
  if (s.rows == 32) return launch_short_variant<2, false>(p, maps, C, stream);
  return launch_short_variant<4, false>(p, maps, C, stream);
}

}  // namespace mla
