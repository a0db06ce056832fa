// FP8 products of a few rows (decode), dense or routed to experts by offsets (sm_103a): the gated feed-forward's
// hidden layer (formulas: gate.cuh), with a scale per row or per block of 128, and the block-scaled product.
//
// With a few rows the work is reading the weights once; the tile kernel (gemm_kernel.cuh) gives a CTA 256 columns of the
// output, which leaves most SMs idle where the output is narrow, and reads the weights through N = 256 MMAs whose M is
// nearly empty. Here:
//  - The weights are the MMA's M side (128 rows a tile; gated: 128 of the gate and the same 128 of the up projection, each
//    with an accumulator of its own, so that both values of an element meet in one thread), the rows its N: 16, 32 or
//    64 of them. Experts with more take several tiles.
//  - Where there are fewer tiles than SMs, a cluster of 2 or 4 CTAs shares a tile's contraction: each leaves its
//    fp32 sums in shared memory and takes a share of the tile's rows to add them up, in the CTAs' order, so that the
//    result is the same on every run.
//  - One K block of 128 a ring stage: the weights' 16 or 32 KB by TMA, past L2's other lines, and the rows' codes.
//  - Blockwise: each K block goes to a fresh tensor-memory partial, and the four epilogue warps (a thread per weight row)
//    add it to their registers, scaled by sA[row, kb] * sB[block, kb] from shared memory, where the epilogue's threads
//    put those products eight K blocks at a time, loaded eight ahead.
// Warps: 0 TMA producer, 1 MMA issuer, 2 .. 5 epilogue. Every wait is bounded; on a timeout the kernel raises
// FP8_DEV_TIMEOUT, drains its loads and MMAs, frees its tensor memory and returns.
#include <atomic>

#include "args.h"
#include "common.cuh"
#include "gate.cuh"
#include "internal.h"

namespace fp8lin {

namespace {

constexpr int kRows = 128;  // weight rows of an MMA, output columns of a tile
constexpr int kBox = kRows * 128;
constexpr int kThreads = 192, kEpi0 = 2;
constexpr int kMaxStages = 12, kMaxSplit = 4;
constexpr int kSmemMax = 232448;  // 227 KB a CTA
constexpr int kSmemPair = 115712;  // two CTAs an SM: half of 228 KB less the 1 KB reserved for each
constexpr int kGroup = 8;         // K blocks whose scales are staged together

struct FewParams {
  int64_t M;            // rows
  int N;                // output columns
  uint32_t idesc;
  int nkb, tiles_n;
  int split;            // CTAs of a cluster
  int stages, stage_bytes;
  const int32_t* ends;  // null: dense
  int E;
  const float* sA;
  const float* sB;
  int sa_scalar, sb_scalar;
  GateArgs gate;
  void* out;            // plain: bf16 or fp32 [M, N]
  int out_f32;
  int32_t* status;
  uint64_t wait_ns;
  int test_stall;
};

struct Shared {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t tfull[2], tempty[2];
  uint64_t drain, never;
  uint64_t part_full, part_empty;  // the cluster's sums are there; they have been read
  uint32_t tmem_base;
  int abort;
  uint32_t amax[4][64];            // gated, codes: a row's largest of each warp's 32 columns
};

FP8_DEVI bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, const volatile int* abort, uint64_t limit_ns) {
  const uint64_t t0 = globaltimer();
  for (uint32_t it = 1;; ++it) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
    if ((it & 15u) == 0) {
      if (*abort) return false;
      if (globaltimer() - t0 > limit_ns) return false;
    }
  }
}
FP8_DEVI float ld_cluster(uint32_t addr) {
  float r;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(r) : "r"(addr) : "memory");
  return r;
}
// A tile: 128 output columns from n0 of an expert's rows row0 .. row0 + cnt - 1.
struct FewTile {
  int n0, e, row0, cnt;
};

// GATED: gate and up projection (G = 2), else a plain product (G = 1). BLOCK: block scales. NT: rows of a tile.
template <int GATED, int BLOCK, int NT>
__global__ void __launch_bounds__(kThreads, 1)
    few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA, const FewParams p) {
  constexpr int G = GATED ? 2 : 1;
  constexpr int kBufCols = G * NT;
  constexpr int kTmem = 2 * kBufCols;  // 32 .. 256: a power of two
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* rest = smem + p.stages * p.stage_bytes;
  float* part = reinterpret_cast<float*>(rest);  // [G][NT][128], clusters only
  if (p.split > 1) rest += G * NT * kRows * 4;
  float* scales = reinterpret_cast<float*>(rest);  // [2][kGroup][G][NT], BLOCK
  if (BLOCK) rest += 2 * kGroup * G * NT * 4;
  Shared& S = *reinterpret_cast<Shared*>(rest);
  int32_t* pre = reinterpret_cast<int32_t*>(rest + sizeof(Shared));  // [E + 1]: entries in front of each expert's
  int32_t* beg = pre + p.E + 1;                                      // [E + 1]: its first row
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = p.split > 1 ? (int)cluster_ctarank() : 0;
  const int unit = blockIdx.x / p.split, n_units = gridDim.x / p.split;
  volatile int* abort_flag = &S.abort;
  auto fail = [&]() {
    if (!*abort_flag) {
      *abort_flag = 1;
      set_status(p.status, FP8_DEV_TIMEOUT);
    }
  };

  if (tid == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&S.full[s], 1);
      mbar_init(&S.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&S.tfull[b], 1);
      mbar_init(&S.tempty[b], 4);
    }
    mbar_init(&S.drain, 1);
    mbar_init(&S.never, 1);
    mbar_init(&S.part_full, (uint32_t)(4 * p.split));
    mbar_init(&S.part_empty, (uint32_t)(4 * p.split));
    S.abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmA);
  }
  if (warp == 1) {
    tmem_alloc(&S.tmem_base, kTmem);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_trigger();

  // entries of up to NT rows, by expert
  int entries;
  if (p.ends) {
    int bad = 0;
    for (int e = tid; e < p.E; e += kThreads) {
      const int32_t cur = ld_l2(p.ends + e), prev = e ? ld_l2(p.ends + e - 1) : 0;
      if (cur < prev || prev < 0 || (e == p.E - 1 && cur != p.M)) bad = 1;
      pre[e + 1] = cur > prev ? (cur - prev + NT - 1) / NT : 0;
      beg[e + 1] = cur;
    }
    if (tid == 0) pre[0] = beg[0] = 0;
    bad = __syncthreads_or(bad);
    if (bad) {  // all CTAs of a cluster see the same offsets and leave together
      if (blockIdx.x == 0 && tid == 0) set_status(p.status, FP8_DEV_BAD_OFFSETS);
      if (warp == 1) tmem_dealloc(S.tmem_base, kTmem);
      return;
    }
    if (warp == 0) {
      int carry = 0;
      for (int base = 0; base < p.E; base += 32) {
        const int i = base + lane;
        int v = i < p.E ? pre[i + 1] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, v, o);
          if (lane >= o) v += y;
        }
        if (i < p.E) pre[i + 1] = v + carry;
        carry += __shfl_sync(0xffffffffu, v, 31);
      }
    }
    tc_fence_before();
    __syncthreads();
    entries = pre[p.E];
  } else {
    entries = (int)((p.M + NT - 1) / NT);
    tc_fence_before();
    __syncthreads();
  }
  if (p.split > 1) cluster_barrier();  // the peers' barriers are initialised before any remote use
  tc_fence_after();
  const uint32_t tmem_base = S.tmem_base;
  const int total = entries * p.tiles_n;
  const int k0 = p.nkb * rank / p.split, k1 = p.nkb * (rank + 1) / p.split;  // this CTA's K blocks

  auto tile = [&](int t) {
    FewTile T;
    const int a = t / p.tiles_n;
    T.n0 = (t - a * p.tiles_n) * kRows;
    T.e = 0;
    T.row0 = a * NT;
    int end = (int)p.M;
    if (p.ends) {
      int lo = 0, hi = p.E - 1;  // the last expert whose entries begin at or before a
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (pre[mid] <= a) lo = mid;
        else hi = mid - 1;
      }
      T.e = lo;
      T.row0 = beg[lo] + (a - pre[lo]) * NT;
      end = beg[lo + 1];
    }
    T.cnt = end - T.row0 < NT ? end - T.row0 : NT;
    return T;
  };

  if (warp == 0) {
    // ================================ TMA producer ================================
    if (lane == 0) {
      const uint64_t pol = l2_evict_first();
      int s = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = unit; t < total && ok; t += n_units) {
        const FewTile T = tile(t);
        for (int kb = k0; kb < k1; ++kb) {
          if (!mbar_wait(&S.empty[s], phase ^ 1, abort_flag, p.wait_ns)) {
            fail();
            ok = false;
            break;
          }
          uint8_t* w = smem + s * p.stage_bytes;
          mbar_arrive_expect_tx(&S.full[s], (uint32_t)(G * kBox + NT * 128));
          tma_load_3d_hint(w, &tmW, &S.full[s], kb * 128, T.n0, G * T.e, pol);  // gated: a box of both projections
          tma_load_2d(w + G * kBox, &tmA, &S.full[s], kb * 128, T.row0);
          ++issued;
          if (++s == p.stages) s = 0, phase ^= 1;
        }
      }
      for (int i = issued > p.stages ? issued - p.stages : 0; i < issued; ++i)  // loads in flight land before exit
        mbar_wait(&S.full[i % p.stages], (uint32_t)((i / p.stages) & 1), nullptr, kDrainNs);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ================================ MMA issuer ================================
    const bool leader = elect_one();
    const uint32_t idesc = p.idesc;
    const uint64_t w_desc0 = smem_desc(smem_u32(smem), 16, 1024);
    bool ok = true;
    if (p.test_stall && !mbar_wait(&S.never, 0, abort_flag, p.wait_ns)) {
      fail();
      ok = false;
    }
    int s = 0, buf = 0;
    uint32_t phase = 0, aphase = 0;
    for (int t = unit; t < total && ok; t += n_units) {
      for (int kb = k0; kb < k1; ++kb) {
        const bool first = BLOCK || kb == k0, last = BLOCK || kb + 1 == k1;  // of what goes to this accumulator
        if (first && !mbar_wait(&S.tempty[buf], aphase ^ 1, abort_flag, p.wait_ns)) {
          fail();
          ok = false;
          break;
        }
        if (!mbar_wait(&S.full[s], phase, abort_flag, p.wait_ns)) {
          fail();
          ok = false;
          break;
        }
        tc_fence_after();
        if (leader) {
          const uint64_t wd = w_desc0 + (uint64_t)((uint32_t)(s * p.stage_bytes) >> 4), ad = wd + (G * kBox >> 4);
          const uint32_t d = tmem_base + (uint32_t)(buf * kBufCols);
#pragma unroll
          for (int g = 0; g < G; ++g)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_f8f6f4(d + g * NT, wd + (uint64_t)(g * (kBox >> 4) + 2 * kk), ad + 2 * kk, idesc,
                          first && kk == 0 ? 0u : 1u);
          umma_commit(&S.empty[s]);
          if (last) umma_commit(&S.tfull[buf]);
        }
        __syncwarp();
        if (++s == p.stages) s = 0, phase ^= 1;
        if (last && ++buf == 2) buf = 0, aphase ^= 1;
      }
    }
    if (leader) umma_commit(&S.drain);
    __syncwarp();
  } else {
    // ================================ epilogue ================================
    const int q = warp & 3, r = q * 32 + lane, etid = tid - 32 * kEpi0;
    const uint32_t lanes = tmem_base + ((uint32_t)(q * 32) << 16);
    const int rows = GATED ? 2 * p.N : p.N, blocks = (rows + kRows - 1) / kRows;  // of an expert's weights
    int buf = 0, sbuf = 0;
    uint32_t aphase = 0, part_phase = 0;
    bool ok = true;
    // the four warps go on or stop together: they meet at named barriers
    auto wait_all = [&](bool got) {
      if (!got) fail();
      return named_bar_and(1, 128, got);
    };
    auto release = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_relaxed(&S.tempty[buf]);
      if (++buf == 2) buf = 0, aphase ^= 1;
    };
    // BLOCK: kGroup K blocks' scales, a thread's share: row j of the tile's and, of every kStep-th K block, the product
    // with either projection's block scale
    constexpr int kStep = 128 / NT, kPer = kGroup / kStep;
    static_assert(kGroup % kStep == 0, "a thread's K blocks of a group");
    const int sj = etid % NT, sk = etid / NT;
    float ra[kPer], rb[G][kPer];
    auto load_scales = [&](const FewTile& T, int kb0) {
      const bool there = sj < T.cnt;
      const float* a = p.sA + (int64_t)(T.row0 + (there ? sj : 0)) * p.nkb;
      const float* b = p.sB + ((int64_t)T.e * blocks + T.n0 / kRows) * p.nkb;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int kb = kb0 + sk + i * kStep;
        const bool live = kb < k1;
        ra[i] = live && there ? ld_l2(a + kb) : 0.f;
#pragma unroll
        for (int g = 0; g < G; ++g) rb[g][i] = live ? ld_l2(b + (int64_t)g * (p.N / kRows) * p.nkb + kb) : 0.f;
      }
    };
    if (BLOCK && unit < total) load_scales(tile(unit), k0);
    for (int t = unit; t < total && ok; t += n_units) {
      const FewTile T = tile(t);
      const int n = T.n0 + r;
      const bool n_ok = n < p.N;
      // rows of this CTA: all of the tile's, or of a cluster's sums rank, rank + split, ...
      const int step = p.split, first = rank;
      // row scales: of the CTA's row j in lane j % 32, and of the thread's weight rows
      float sa[(NT + 31) / 32], sb[G];
      if (!BLOCK) {
#pragma unroll
        for (int i = 0; i < (NT + 31) / 32; ++i) {
          const int row = first + (lane + 32 * i) * step;
          sa[i] = p.sa_scalar ? ld_l2(p.sA) : row < T.cnt ? ld_l2(p.sA + T.row0 + row) : 0.f;
        }
#pragma unroll
        for (int g = 0; g < G; ++g)
          sb[g] = p.sb_scalar ? ld_l2(p.sB) : n_ok ? ld_l2(p.sB + (int64_t)T.e * rows + (int64_t)g * p.N + n) : 0.f;
      }
      float v[G][NT];
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int j = 0; j < NT; ++j) v[g][j] = 0.f;
      if (BLOCK) {
        for (int kb = k0; kb < k1 && ok; ++kb) {
          const int i0 = (kb - k0) & (kGroup - 1);
          if (i0 == 0) {  // the next group's scales into the buffer that the group before the last one used
            sbuf ^= 1;
            float* s = scales + sbuf * (kGroup * G * NT);
#pragma unroll
            for (int i = 0; i < kPer; ++i)
#pragma unroll
              for (int g = 0; g < G; ++g) s[((sk + i * kStep) * G + g) * NT + sj] = ra[i] * rb[g][i];
            named_bar_sync(1, 128);
            if (kb + kGroup < k1)
              load_scales(T, kb + kGroup);
            else if (t + n_units < total)
              load_scales(tile(t + n_units), k0);
          }
          if (!mbar_wait(&S.tfull[buf], aphase, abort_flag, p.wait_ns)) ok = false;
          // at a group's end all warps learn of one that gave up, ahead of the next barrier
          if (i0 == kGroup - 1 || kb + 1 == k1) ok = wait_all(ok);
          if (!ok) {
            if (i0 == kGroup - 1 || kb + 1 == k1) break;
            ok = true;  // the wait's outcome counts at the group's end; the sums no longer do
            fail();
          }
          tc_fence_after();
          const float* s = scales + sbuf * (kGroup * G * NT) + i0 * (G * NT);
          constexpr int W = NT < 32 ? NT : 32;
#pragma unroll
          for (int g = 0; g < G; ++g)
#pragma unroll
            for (int c = 0; c < NT; c += W) {
              uint32_t d[W];
              __syncwarp();
              const uint32_t addr = lanes + (uint32_t)(buf * kBufCols + g * NT + c);
              if constexpr (W == 16) {
                tmem_ld16(addr, d);
                tmem_ld_wait_regs16(d);
              } else {
                tmem_ld32(addr, d);
                tmem_ld_wait_regs(d);
              }
#pragma unroll
              for (int j = 0; j < W; j += 4) {
                const float4 f = *reinterpret_cast<const float4*>(s + g * NT + c + j);
                v[g][c + j] = fmaf(__uint_as_float(d[j]), f.x, v[g][c + j]);
                v[g][c + j + 1] = fmaf(__uint_as_float(d[j + 1]), f.y, v[g][c + j + 1]);
                v[g][c + j + 2] = fmaf(__uint_as_float(d[j + 2]), f.z, v[g][c + j + 2]);
                v[g][c + j + 3] = fmaf(__uint_as_float(d[j + 3]), f.w, v[g][c + j + 3]);
              }
            }
          release();
        }
        if (!ok) break;
      } else {
        if (!wait_all(mbar_wait(&S.tfull[buf], aphase, abort_flag, p.wait_ns))) break;
        tc_fence_after();
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
          for (int c = 0; c < NT; c += 16) {
            uint32_t d[16];
            tmem_ld16(lanes + (uint32_t)(buf * kBufCols + g * NT + c), d);
            tmem_ld_wait_regs16(d);
#pragma unroll
            for (int j = 0; j < 16; ++j) v[g][c + j] = __uint_as_float(d[j]);
          }
        release();
      }
      if (p.split > 1) {  // the CTA's rows of the cluster's sums, moved to the front
        if (!wait_all(mbar_wait_cluster(&S.part_empty, part_phase ^ 1, abort_flag, p.wait_ns))) break;
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
          for (int j = 0; j < NT; ++j)
            if (j < T.cnt) part[(g * NT + j) * kRows + r] = v[g][j];
        __syncwarp();
        if (lane < p.split) mbar_arrive_cluster(mapa_shared(smem_u32(&S.part_full), (uint32_t)lane));
        if (!wait_all(mbar_wait_cluster(&S.part_full, part_phase, abort_flag, p.wait_ns))) break;
        const uint32_t mine = smem_u32(part) + 4 * r;
#pragma unroll
        for (int j0 = 0; j0 < NT / 2; j0 += 8) {
          if (first + j0 * step >= T.cnt) break;
#pragma unroll
          for (int j = j0; j < j0 + 8; ++j)
#pragma unroll
            for (int g = 0; g < G; ++g) v[g][j] = 0.f;
          for (int c = 0; c < p.split; ++c) {
            const uint32_t from = mapa_shared(mine, (uint32_t)c);
#pragma unroll
            for (int j = j0; j < j0 + 8; ++j)
              if (first + j * step < T.cnt)
#pragma unroll
                for (int g = 0; g < G; ++g) v[g][j] += ld_cluster(from + (uint32_t)((g * NT + first + j * step) * (kRows * 4)));
          }
        }
        __syncwarp();
        if (lane < p.split) mbar_arrive_cluster(mapa_shared(smem_u32(&S.part_empty), (uint32_t)lane));
        part_phase ^= 1;
      }
      // eight rows at a time, without a branch between them, so that their latencies overlap
#pragma unroll
      for (int j0 = 0; j0 < NT; j0 += 8) {
        if (first + j0 * step >= T.cnt) break;
        if (!BLOCK) {  // (acc * sA[row]) * sB[column], as the tile kernel rounds
#pragma unroll
          for (int j = j0; j < j0 + 8; ++j) {
            const float s = __shfl_sync(0xffffffffu, sa[j / 32], j % 32);
#pragma unroll
            for (int g = 0; g < G; ++g) v[g][j] = v[g][j] * s * sb[g];
          }
        }
        if constexpr (!GATED) {
#pragma unroll
          for (int j = j0; j < j0 + 8; ++j) {
            const int row = first + j * step;
            const int64_t at = (int64_t)(T.row0 + row) * p.N + n;
            const bool put = n_ok && row < T.cnt;
            if (put && p.out_f32)
              static_cast<float*>(p.out)[at] = v[0][j];
            else if (put)
              static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(v[0][j]);
          }
        } else {
          if (p.gate.gu) {
#pragma unroll
            for (int j = j0; j < j0 + 8; ++j) {
              const int row = first + j * step;
              __nv_bfloat16* o = p.gate.gu + (int64_t)(T.row0 + row) * 2 * p.N + n;
              if (n_ok && row < T.cnt) {
                o[0] = __float2bfloat16_rn(v[0][j]);
                o[p.N] = __float2bfloat16_rn(v[G - 1][j]);
              }
            }
          }
          gate_fwd<8>(p.gate.act, v[0] + j0, v[G - 1] + j0, v[0] + j0);
          if (p.gate.h) {
#pragma unroll
            for (int j = j0; j < j0 + 8; ++j) {
              const int row = first + j * step;
              if (n_ok && row < T.cnt) p.gate.h[(int64_t)(T.row0 + row) * p.N + n] = __float2bfloat16_rn(v[0][j]);
            }
          }
          if (p.gate.q) {  // bit patterns of magnitudes order as the magnitudes, a NaN's above all
#pragma unroll
            for (int j = j0; j < j0 + 8; ++j) {
              const uint32_t am = __reduce_max_sync(0xffffffffu, __float_as_uint(v[0][j]) & 0x7FFFFFFFu);
              if (lane == 0) S.amax[q][j] = am;
            }
          }
        }
      }
      if (GATED && p.gate.q) {  // N % 128 == 0: the tile's columns are one whole block
        named_bar_sync(1, 128);
        const bool e4 = p.gate.q_fmt == FP8_DT_E4M3;
#pragma unroll
        for (int j0 = 0; j0 < NT; j0 += 8) {
          if (first + j0 * step >= T.cnt) break;
#pragma unroll
          for (int j = j0; j < j0 + 8; ++j) {
            const int row = first + j * step;
            const int64_t m = T.row0 + row;
            const float a = max_nan(__uint_as_float(max(max(S.amax[0][j], S.amax[1][j]), max(S.amax[2][j], S.amax[3][j]))),
                                    (float)kEps);
            const float x = v[0][j] * __fdiv_rn(e4 ? kE4M3Max : kE5M2Max, a);
            const uint8_t code = (uint8_t)(e4 ? cvt_fp8x2<FP8_DT_E4M3>(x, 0.f) : cvt_fp8x2<FP8_DT_E5M2>(x, 0.f));
            if (row < T.cnt) {
              p.gate.q[m * p.N + n] = code;
              if (etid == 0) p.gate.inv[m * (p.N / kRows) + T.n0 / kRows] = a * (e4 ? 1.0f / kE4M3Max : 1.0f / kE5M2Max);
            }
          }
        }
        named_bar_sync(1, 128);  // read before the next tile's are written
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (p.split > 1) cluster_barrier();  // no remote access to a CTA that has left
  if (warp == 1) {
    if (lane == 0) mbar_wait(&S.drain, 0, nullptr, kDrainNs);  // the MMAs that write tensor memory
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, kTmem);
  }
}

template <int GATED, int BLOCK, int NT>
int run_few(const CUtensorMap& tw, const CUtensorMap& ta, FewParams p, int64_t tiles, const Ctx& c) {
  constexpr int G = GATED ? 2 : 1;
  auto kern = few_kernel<GATED, BLOCK, NT>;
  static std::atomic<uint64_t> done{0};
  const uint64_t bit = 1ull << (c.device & 63);
  if (!(done.load(std::memory_order_acquire) & bit)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax) != cudaSuccess)
      return FP8_ERR_CUDA;
    done.fetch_or(bit, std::memory_order_release);
  }
  // Fewer tiles than SMs: 2 or 4 CTAs share one's contraction, as long as all clusters run at once (one token of 7168 x
  // 2048, 16 tiles: 21 us alone, 14 in twos, 11 in fours, 18 in eights, of which few fit the GPU at a time; 4096 x
  // 14336, 112 tiles: 22 and 23, 34 in fours).
  p.split = 1;
  while (p.split < kMaxSplit && 2 * tiles * p.split * 16 <= (int64_t)c.sm_count * 15 && p.nkb >= 4 * p.split) p.split *= 2;
  p.stage_bytes = G * kBox + NT * 128;
  const int rest = 1024 + (p.split > 1 ? G * NT * kRows * 4 : 0) + (BLOCK ? 2 * kGroup * G * NT * 4 : 0) +
                   (int)sizeof(Shared) + 8 * (p.E + 1);
  // Where half an SM's shared memory holds four stages or more, the ring takes no more, and the next call's CTAs start
  // up beside this one's (8 experts of 2048 x 7168, one row each: 25.1 to 23.9 us; three stages of the gated
  // product in it, 22.6 us for 4096 x 14336, against six alone, 22.0).
  const int pair = (kSmemPair - rest) / p.stage_bytes;
  const int fit = pair >= 4 ? pair : (kSmemMax - rest) / p.stage_bytes;
  p.stages = fit < kMaxStages ? fit : kMaxStages;
  const int64_t units = c.sm_count / p.split;
  const int64_t grid = (tiles < units ? tiles : units) * p.split;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)p.split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)(rest + p.stages * p.stage_bytes);
  cfg.stream = c.stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, tw, ta, p) == cudaSuccess ? FP8_OK : FP8_ERR_CUDA;
}

template <int GATED, int BLOCK>
int by_rows(const CUtensorMap& tw, const CUtensorMap& ta, const FewParams& p, int nt, int64_t tiles, const Ctx& c) {
  return nt == 16   ? run_few<GATED, BLOCK, 16>(tw, ta, p, tiles, c)
         : nt == 32 ? run_few<GATED, BLOCK, 32>(tw, ta, p, tiles, c)
                    : run_few<GATED, BLOCK, 64>(tw, ta, p, tiles, c);
}

}  // namespace

// nt: rows of a tile, the smallest of 16, 32 and 64 that holds them all.
static int launch_few(const void* A, const void* B, int a_dtype, int b_dtype, int64_t M, int64_t N, int64_t K, int64_t E,
                      bool gated, bool block, FewParams& p, const Ctx& c) {
  const int nt = M <= 16 ? 16 : M <= 32 ? 32 : 64;
  const int G = gated ? 2 : 1;
  p.M = M;
  p.N = (int)N;
  p.E = (int)E;
  p.nkb = (int)ceil_div64(K, 128);
  p.tiles_n = (int)ceil_div64(N, kRows);
  p.status = c.status;
  p.wait_ns = c.wait_ns;
  p.test_stall = c.test_stall;
  p.idesc = make_idesc(b_dtype == FP8_DT_E4M3 ? kFmtE4M3 : kFmtE5M2, a_dtype == FP8_DT_E4M3 ? kFmtE4M3 : kFmtE5M2, 0,
                            0, kRows, (uint32_t)nt);
  const int64_t n_exp = E ? E : 1;
  // at most: no more experts than rows have any, and the last entry of each may be part empty
  const int64_t entries = ceil_div64(M, nt) + (p.ends ? (M < n_exp ? M : n_exp) - 1 : 0);
  if (entries * p.tiles_n >= (int64_t)1 << 31) return FP8_ERR_UNSUPPORTED;
  CUtensorMap tw, ta;
  {
    const uint64_t d[3] = {(uint64_t)K, (uint64_t)N, (uint64_t)(G * n_exp)}, st[2] = {(uint64_t)K, (uint64_t)(N * K)};
    const uint32_t box[3] = {128, kRows, (uint32_t)G};
    FP8_TRY(make_tmap(&tw, B, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, d, st, box, CU_TENSOR_MAP_SWIZZLE_128B));
  }
  {
    const uint64_t d[2] = {(uint64_t)K, (uint64_t)M}, st[1] = {(uint64_t)K};
    const uint32_t box[2] = {128, (uint32_t)nt};
    FP8_TRY(make_tmap(&ta, A, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, d, st, box, CU_TENSOR_MAP_SWIZZLE_128B));
  }
  const int64_t tiles = entries * p.tiles_n;
  if (!gated) return by_rows<0, 1>(tw, ta, p, nt, tiles, c);
  return block ? by_rows<1, 1>(tw, ta, p, nt, tiles, c) : by_rows<1, 0>(tw, ta, p, nt, tiles, c);
}

int launch_few_gated(const GatedArgs& g, const Ctx& c) {
  FewParams p = {};
  p.ends = g.ends;
  p.sA = g.sA;
  p.sB = g.sB;
  p.sa_scalar = g.sa_scalar;
  p.sb_scalar = g.sb_scalar;
  p.gate.act = g.act;
  p.gate.gu = static_cast<__nv_bfloat16*>(g.gu);
  p.gate.h = static_cast<__nv_bfloat16*>(g.h);
  p.gate.q = static_cast<uint8_t*>(g.q);
  p.gate.inv = g.inv;
  p.gate.q_fmt = g.q_fmt;
  return launch_few(g.A, g.B, g.a_dtype, g.b_dtype, g.M, g.I, g.K, g.E, true, g.blockwise != 0, p, c);
}

int launch_few_blockwise(const GemmArgs& g, const Ctx& c) {
  FewParams p = {};
  p.ends = g.ends;
  p.sA = g.sA;
  p.sB = g.sB;
  p.out = g.out;
  p.out_f32 = g.out_dtype == FP8_DT_F32;
  return launch_few(g.A, g.B, g.a_dtype, g.b_dtype, g.M, g.N, g.K, g.E, false, true, p, c);
}

}  // namespace fp8lin
