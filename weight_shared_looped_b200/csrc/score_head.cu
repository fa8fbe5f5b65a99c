// Scoring head: log probabilities of given tokens under the logits
// z[v] = y . E[v] (fp32 activations y, fp16 embedding rows E[v]), the entropy of
// each row's distribution and its k most probable tokens.  The logits are never
// stored:
//   lse = log sum_v exp(z[v]),   logp(t) = z[t] - lse,
//   entropy = lse - sum_v exp(z[v] - lse) z[v]
//
// Pass 0 splits the activations of each row, scaled by a power of two so that
// the row's largest lies in [2^9, 2^10), into two fp16 parts, y = hi + lo: 22 bits
// of each activation, and no row over- or underflows.  Both parts meet the same
// embedding tile on the tensor cores, for twice the matrix work (one fp16 part alone
// would leave errors of 2^-12 per activation in every probability).
//
// The tensor cores add towards zero.  An addition loses up to 2^-23 of the sum so far, half
// of that on average, always to the same side, so the loss does not average out over the
// vocabulary as an fp32 sum's roundings do, and it depends on where along d a logit comes
// from, so no factor takes it back.  The accumulators therefore hold SC_CHUNK k blocks at a
// time, and their sums are added in fp32.  Chunks of 2048, 1024, 512, 256 and 128 elements
// leave rows of d 2048 whose logits of 32 come from one early channel off by 2.8e-4, 1.3e-4,
// 6.6e-5, 3.1e-5 and 1.4e-5 (row-major; half of it vocabulary-major); 1021 rows with k 3 take
// 303, 309, 312, 334 and 369 us, 56 rows with k 5 64, 65, 68, 75 and 81.  Chunks of 512 are
// the shortest that the epilogue keeps up with.
//
// Pass 1 streams the embedding through tcgen05 and keeps, per row and slice of
// the vocabulary, the running maximum m, l = sum e^(z - m), s = sum e^(z - m) (z - m)
// and the best candidates.
// Pass 2, a CTA per row (a warp per row where there are many), merges the slices and
// decides the order of the best k + kSpare candidates, and the given token's logit, by
// fp64 dot products of the inputs (ties go to the lowest token id; equal embedding rows
// tie in pass 1 already, and for another token to be missed, three logits have to lie
// within pass 1's error of the k-th: it is then as good to that error).
//
// Bounds (vocabulary 50257, d 2048): few rows by the embedding's 206 MB, 31 us; one row
// with k 5 takes 46 us (passes 0 and 2 and the fill and tail of pass 1 are 12 of
// them).  Many rows by the matrix work, twice 2 n V d; 1021 rows with k 3 in 311 us,
// 1.35 PFLOP/s.  In between the epilogue of the last tiles shows: 128 rows with k 8 take
// 82 us.
#include <math_constants.h>

#include <algorithm>
#include <cstring>

#include "tc_util.cuh"

namespace tl {
namespace {

constexpr int kSpare = 2;          // candidates scored in fp64 beyond k
constexpr int kMaxCand = 20;       // candidates kept per slice, at most
constexpr int SC_BK = 64;          // k per stage (one 128-byte swizzled row)
constexpr int SC_CHUNK = 8;        // k blocks of one accumulator: see above
static_assert(SC_CHUNK % 2 == 0, "whole stages of up to two k blocks");
constexpr int kScoreSms = 148;

__device__ __forceinline__ bool sc_better(float x, int v, float bx, int bv) {
  return x > bx || (x == bx && v < bv);
}

// Slice records: stat[row][slice] = (m, l, s) in base 2 (s in units of log2);
// top_x, top_v[row][rank][slice] = the slice's best kc candidates by rank.
struct ScoreRec {
  float4* stat;
  float* top_x;
  int* top_v;
};

// the largest float below x (x not NaN)
__device__ __forceinline__ float sc_below(float x) {
  if (x == -INFINITY) return x;
  const int u = __float_as_int(x);
  return __int_as_float(x > 0.f ? u - 1 : x < 0.f ? u + 1 : (int)0x80000001);
}

__device__ __forceinline__ float sc_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ------------------------------------------------------------------ pass 0
// One CTA per row of the padded batch: parts[row] = hi, parts[pad + row] = lo
// (zeros behind the batch), scale[row] = the power of two taken out.
__global__ void __launch_bounds__(256) score_split_kernel(const float* __restrict__ y, long y_stride, int n, int d,
                                                          int pad, __half* parts, float* scale, int* clear) {
  pdl_enter();
  __shared__ float wmax[8];
  const int row = blockIdx.x, tid = threadIdx.x;
  if (row == 0 && tid == 0 && clear) *clear = 0;
  __half* hi = parts + (size_t)row * d;
  __half* lo = parts + (size_t)(pad + row) * d;
  if (row >= n) {
    for (int i = tid * 4; i < d; i += 1024) {
      *reinterpret_cast<uint2*>(hi + i) = make_uint2(0u, 0u);
      *reinterpret_cast<uint2*>(lo + i) = make_uint2(0u, 0u);
    }
    return;
  }
  const float* yr = y + (size_t)row * y_stride;
  float4 v[8];                     // d <= 8192
  float mx = 0.f;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int i = (tid + u * 256) * 4;
    if (i < d) {
      v[u] = *reinterpret_cast<const float4*>(yr + i);
      mx = fmaxf(mx, fmaxf(fmaxf(fabsf(v[u].x), fabsf(v[u].y)), fmaxf(fabsf(v[u].z), fabsf(v[u].w))));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if ((tid & 31) == 0) wmax[tid >> 5] = mx;
  __syncthreads();
  for (int w = 0; w < 8; ++w) mx = fmaxf(mx, wmax[w]);
  // 2^e <= mx < 2^(e + 1); rows of zeros or with an infinity are taken as they are
  int e = 9;
  if (mx > 0.f && mx < CUDART_INF_F) e = ilogbf(mx);
  e = max(e, -117);                // 2^(9 - e) stays finite; smaller rows keep fewer bits of tiny logits
  const float mul = ldexpf(1.f, 9 - e);
  if (tid == 0) scale[row] = ldexpf(1.f, e - 9);
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int i = (tid + u * 256) * 4;
    if (i < d) {
      const float f[4] = {v[u].x * mul, v[u].y * mul, v[u].z * mul, v[u].w * mul};
      __half h[4], l[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        h[q] = __float2half_rn(f[q]);
        l[q] = __float2half_rn(f[q] - __half2float(h[q]));
      }
      *reinterpret_cast<uint2*>(hi + i) = *reinterpret_cast<uint2*>(h);
      *reinterpret_cast<uint2*>(lo + i) = *reinterpret_cast<uint2*>(l);
    }
  }
}

// ------------------------------------------------------------------ pass 1
// One thread issues the copies and one the MMAs: a lone lane has its SM
// sub-partition nearly to itself here, and its loop is shorter than a converged
// warp's with an election per instruction (a stage took 830 cycles that way,
// waits included, however small its copies).
__device__ __forceinline__ void sc_mma(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void sc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void sc_expect(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void sc_copy(uint64_t* bar, void* dst, const CUtensorMap* map, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%1], [%2, {%3, %4}], [%0];" ::"r"(
          smem_u32(bar)),
      "r"(smem_u32(dst)), "l"(map), "r"(x), "r"(y)
      : "memory");
}
// a bounded wait by one thread; false once it ran out or another role gave up
__device__ __forceinline__ bool sc_wait(uint64_t* bar, uint32_t parity, const int* abort_flag, uint64_t limit_ns) {
  if (mbar_try(smem_u32(bar), parity)) return true;
  return mbar_wait(bar, parity, limit_ns) && !*(volatile const int*)abort_flag;
}

__device__ __forceinline__ void sc_ld16(uint32_t* u, uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
        "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
      : "r"(addr));
}
// the wait carries the registers, so that no use of them moves above it
__device__ __forceinline__ void sc_ld_wait(uint32_t* u) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(u[0]), "+r"(u[1]), "+r"(u[2]), "+r"(u[3]), "+r"(u[4]), "+r"(u[5]), "+r"(u[6]), "+r"(u[7]),
                 "+r"(u[8]), "+r"(u[9]), "+r"(u[10]), "+r"(u[11]), "+r"(u[12]), "+r"(u[13]), "+r"(u[14]), "+r"(u[15])
               :
               : "memory");
}
// keeps uses of registers that an earlier wait covers below it
__device__ __forceinline__ void sc_pin16(uint32_t* u) {
  asm volatile(""
               : "+r"(u[0]), "+r"(u[1]), "+r"(u[2]), "+r"(u[3]), "+r"(u[4]), "+r"(u[5]), "+r"(u[6]), "+r"(u[7]),
                 "+r"(u[8]), "+r"(u[9]), "+r"(u[10]), "+r"(u[11]), "+r"(u[12]), "+r"(u[13]), "+r"(u[14]), "+r"(u[15]));
}
// barrier 1 over the eight statistics warps; true for all when `bad` is for any
__device__ __forceinline__ bool sc_barrier_or(bool bad) {
  uint32_t any;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 q, %1, 0;\n barrier.cta.red.or.pred p, 1, 256, q;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(any)
      : "r"(bad ? 1u : 0u)
      : "memory");
  return any != 0;
}

struct ScoreTc {
  int n, V, nkb;          // rows, vocabulary, k blocks
  int pad;                // rows of one activation part
  int bn;                 // vocabulary entries per tile
  int vt;                 // tiles of the vocabulary
  int mt, groups;         // row tiles; CTAs that share one row tile's vocabulary tiles
  int stages;
  uint32_t stage_bytes;
  int slices;             // records per row
  int slots;              // vocabulary-major: accumulators in TMEM
  const float* scale;
  ScoreRec rec;
  int* flag;              // takes kDevTimeout when a bounded wait ran out
  uint64_t wait_ns;       // limit of a wait
  int copies;             // stages that the copying thread fills at most (a test of the waits fills too few)
};

constexpr int SC_SLOTS = 8;        // accumulators of a CTA, at most
constexpr float kLog2e = 1.4426950408889634f;

struct ScoreBars {
  uint64_t full[12], empty[12], acc_full[SC_SLOTS], acc_empty[SC_SLOTS];
  uint64_t drained;
  uint32_t tmem;
  int abort, issued;      // a role gave up; stages requested
};

// After the roles have met: where one gave up, the copies and MMAs still in flight end
// before the CTA leaves and gives back its TMEM (threads 256 and 288 issued them).
__device__ __forceinline__ void sc_settle(ScoreBars& bars, int stages, int* flag) {
  if (!bars.abort) return;
  if (threadIdx.x == 256)
    for (int i = max(0, bars.issued - stages); i < bars.issued; ++i) mbar_wait(&bars.full[i % stages], (i / stages) & 1);
  if (threadIdx.x == 288) {
    sc_commit(&bars.drained);
    mbar_wait(&bars.drained, 0);
  }
  if (threadIdx.x == 0) atomicExch(flag, kDevTimeout);
  __syncwarp();
  __syncthreads();
}

// Row-major variant: 128 rows of activations (hi and lo) are the MMA's M side,
// bn vocabulary entries its N side, so an epilogue thread owns one row and walks
// its logits: the softmax statistics and the candidate list live in registers.
// Warps 0-7 read the accumulators (warp w: TMEM quadrant w mod 4, column half
// w / 4) and add up a tile's chunks, warp 8 copies, warp 9 issues the MMAs; two
// accumulators of 256 columns let the epilogue of one tile run under the next
// tile's MMAs.
constexpr int SR_THREADS = 384;    // three warpgroups; the last one's other two warps idle
// A statistics thread holds the 128 logits of its half tile, so that an accumulator is free
// again once it is read; its warpgroups take registers that the issuing one gives up.
constexpr int SR_REGS = 168;       // a thread's registers at launch: the launch bounds' share of the SM
constexpr int SR_REGS_STAT = 232, SR_REGS_ISSUE = 40;
static_assert(2 * SR_REGS_STAT + SR_REGS_ISSUE <= 3 * SR_REGS, "no more than the block was launched with");
constexpr int SR_QUEUE = 16;       // newcomers a statistics thread can hold

// A logit above `bar` goes to the queue at `at`, whose entries are 256 threads apart.
// (Written out: the compiler branches around the store.)
__device__ __forceinline__ void sc_push(uint32_t& at, float x, float bar, int id) {
  asm volatile(
      "{\n .reg .pred p;\n setp.gt.f32 p, %1, %2;\n @p st.shared.v2.b32 [%0], {%3, %4};\n"
      " @p add.u32 %0, %0, 2048;\n}\n"
      : "+r"(at)
      : "f"(x), "f"(bar), "r"(__float_as_uint(x)), "r"(id)
      : "memory");
}

template <int KC>
__global__ void __launch_bounds__(SR_THREADS, 1)
    score_rows_kernel(const __grid_constant__ CUtensorMap map_y, const __grid_constant__ CUtensorMap map_e, ScoreTc a) {
  extern __shared__ uint8_t sr_raw[];
  __shared__ ScoreBars bars;
  uint8_t* smem = (uint8_t*)(((uintptr_t)sr_raw + 1023) & ~(uintptr_t)1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // row tile blockIdx.x mod mt, every groups-th vocabulary tile: the CTAs of one
  // group read the same embedding tile together, so it leaves HBM once
  const int mt = blockIdx.x % a.mt, group = blockIdx.x / a.mt;
  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(&bars.full[s], 1);
      mbar_init(&bars.empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars.acc_full[s], 1);
      mbar_init(&bars.acc_empty[s], 8);
    }
    mbar_init(&bars.drained, 1);
    bars.abort = bars.issued = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncwarp();
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&bars.tmem)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = bars.tmem;
  pdl_enter();

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(SR_REGS_ISSUE));
    if (warp == 8) {
      // ---------------------------------------------------------------- copies
      if (lane == 0) {
        int s = 0, ph = 1, issued = 0;
        bool ok = true;
        const int r0 = mt * 128;
        for (int vt = group; vt < a.vt && ok; vt += a.groups) {
          const int v0 = vt * a.bn;
          for (int kb = 0; kb < a.nkb && issued < a.copies; ++kb) {
            if (issued >= a.stages && !sc_wait(&bars.empty[s], ph, &bars.abort, a.wait_ns)) {
              ok = false;
              break;
            }
            uint8_t* st = smem + (size_t)s * a.stage_bytes;
            sc_expect(&bars.full[s], a.stage_bytes);
            sc_copy(&bars.full[s], st, &map_y, kb * SC_BK, r0);
            sc_copy(&bars.full[s], st + 16384, &map_y, kb * SC_BK, a.pad + r0);
            sc_copy(&bars.full[s], st + 32768, &map_e, kb * SC_BK, v0);
            ++issued;
            if (++s == a.stages) {
              s = 0;
              ph ^= 1;
            }
          }
        }
        if (!ok) atomicExch(&bars.abort, 1);
        bars.issued = issued;
      }
      __syncwarp();
    } else if (warp == 9) {
      // ---------------------------------------------------------------- MMAs
      if (lane == 0) {
        const uint32_t idesc = (1u << 4) | ((uint32_t)(a.bn >> 3) << 17) | (8u << 24);
        const uint64_t desc0 = smem_desc_sw128(smem_u32(smem));   // + stage bytes / 16 per stage: stays below 2^14
        int s = 0, ph = 0, i = 0;
        bool ok = true;
        for (int vt = group; vt < a.vt && ok; vt += a.groups) {
          for (int k0 = 0; k0 < a.nkb && ok; k0 += SC_CHUNK, ++i) {
            const int buf = i & 1, use = i >> 1;
            if (use > 0) ok = sc_wait(&bars.acc_empty[buf], (use & 1) ^ 1, &bars.abort, a.wait_ns);
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t acc = tmem + buf * 256;
            for (int kb = k0; kb < min(k0 + SC_CHUNK, a.nkb) && ok; ++kb) {
              ok = sc_wait(&bars.full[s], ph, &bars.abort, a.wait_ns);
              if (!ok) break;
              asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
              const uint64_t hi = desc0 + (uint64_t)(s * (a.stage_bytes >> 4)), lo = hi + (16384 >> 4), e = hi + (32768 >> 4);
              // the small parts first: their additions lose next to nothing in an empty accumulator
#pragma unroll
              for (int ks = 0; ks < 4; ++ks) sc_mma(acc, lo + 2 * ks, e + 2 * ks, idesc, kb != k0 || ks != 0);
#pragma unroll
              for (int ks = 0; ks < 4; ++ks) sc_mma(acc, hi + 2 * ks, e + 2 * ks, idesc, true);
              sc_commit(&bars.empty[s]);
              if (++s == a.stages) {
                s = 0;
                ph ^= 1;
              }
            }
            if (ok) sc_commit(&bars.acc_full[buf]);
          }
        }
        if (!ok) atomicExch(&bars.abort, 1);
      }
      __syncwarp();
    }
  } else {
    // ---------------------------------------------------------------- statistics
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(SR_REGS_STAT));
    const int half = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t laddr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const int cols = a.bn / 2;                         // a multiple of 16
    const int row = mt * 128 + r;
    const float rs = row < a.n ? a.scale[row] : 1.f, rs2 = rs * kLog2e;
    float m = -INFINITY, l = 0.f, sx = 0.f;            // in log2 units
    // the row's best so far, and a queue of newcomers in shared memory: logits
    // above the list's last are queued (a predicated store each) and inserted when
    // some lane's queue fills, so the insertion network runs about as often as the
    // busiest lane needs, not as often as any lane does
    float cx[KC];
    int cv[KC];
#pragma unroll
    for (int p = 0; p < KC; ++p) {
      cx[p] = -INFINITY;
      cv[p] = 0x7fffffff;
    }
    const uint32_t queue = smem_u32(smem + (size_t)a.stages * a.stage_bytes) + 8 * threadIdx.x;   // [SR_QUEUE][256]
    uint32_t at = queue;
    auto drain = [&]() {
      const uint32_t end = __reduce_max_sync(0xffffffffu, at - queue) + queue;
#pragma unroll 1
      for (uint32_t q = queue; q < end; q += 2048) {
        uint32_t xb, id;
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(xb), "=r"(id) : "r"(q) : "memory");
        const float xv = q < at ? __uint_as_float(xb) : -INFINITY;
        // an equal entry seen earlier (a lower id) stays before
#pragma unroll
        for (int p = KC - 1; p > 0; --p) {
          const bool up = xv > cx[p - 1], in = xv > cx[p];
          cv[p] = up ? cv[p - 1] : in ? (int)id : cv[p];
          cx[p] = up ? cx[p - 1] : in ? xv : cx[p];
        }
        if (xv > cx[0]) {
          cx[0] = xv;
          cv[0] = (int)id;
        }
      }
      at = queue;
    };
    bool ok = true;
    int i = 0;
    uint32_t z[128];                                   // the tile's logits (fp32)
    for (int vt = group; vt < a.vt && ok; vt += a.groups) {
      for (int k0 = 0; k0 < a.nkb; k0 += SC_CHUNK, ++i) {
        const int buf = i & 1, use = i >> 1;
        if (!warp_wait(&bars.acc_full[buf], use & 1, &bars.abort, true, a.wait_ns)) {
          if (lane == 0) atomicExch(&bars.abort, 1);
          ok = false;
          break;
        }
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t base = laddr + buf * 256 + half * cols;
        if (k0 == 0) {
#pragma unroll
          for (int b = 0; b < 8; ++b)
            if (16 * b < cols) sc_ld16(z + 16 * b, base + 16 * b);
          sc_ld_wait(z);
#pragma unroll
          for (int b = 1; b < 8; ++b) sc_pin16(z + 16 * b);
        } else {
          uint32_t w[2][16];
          sc_ld16(w[0], base);
#pragma unroll
          for (int b = 0; b < 8; ++b) {
            if (16 * b < cols) {
              sc_ld_wait(w[b & 1]);
              if (16 * b + 16 < cols) sc_ld16(w[(b & 1) ^ 1], base + 16 * b + 16);
#pragma unroll
              for (int j = 0; j < 16; ++j)
                z[16 * b + j] = __float_as_uint(__uint_as_float(z[16 * b + j]) + __uint_as_float(w[b & 1][j]));
            }
          }
        }
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.acc_empty[buf]);
      }
      if (!ok) break;
      const int v0 = vt * a.bn + half * cols;
      const int valid = min(cols, a.V - v0);           // may be <= 0 in the last tile
      // 32 logits, z[z0] and on; two chains of sums, so that they wait less for each other
      auto take = [&](int c, int z0) {
        const int nv = min(cols, valid) - c;           // uniform over the warp
        if (nv <= 0) return;
        if (nv < 32)
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (j >= nv) z[z0 + j] = 0xff800000u;           // below every logit
        auto x = [&](int j) { return __uint_as_float(z[z0 + j]); };
        float top4[4] = {x(0), x(1), x(2), x(3)};
#pragma unroll
        for (int j = 4; j < 32; ++j) top4[j & 3] = fmaxf(top4[j & 3], x(j));
        const float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3]));
        const float top2 = top * rs2;
        if (top2 > m) {
          const float f = sc_ex2(m - top2);
          sx = l == 0.f ? 0.f : (sx + l * (m - top2)) * f;
          l *= f;
          m = top2;
        }
        float l2[2] = {0.f, 0.f}, s2[2] = {0.f, 0.f};
        if (nv >= 32) {
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float t = fmaf(x(j), rs2, -m), e = sc_ex2(t);
            l2[j & 1] += e;
            s2[j & 1] = fmaf(e, t, s2[j & 1]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) {               // e = 0 where there is no logit
            const float t = j < nv ? fmaf(x(j), rs2, -m) : -1e4f, e = sc_ex2(t);
            l2[j & 1] += e;
            s2[j & 1] = fmaf(e, t, s2[j & 1]);
          }
        }
        l += l2[0] + l2[1];
        sx += s2[0] + s2[1];
        if (__any_sync(0xffffffffu, top > cx[KC - 1])) {
          const int id = v0 + c;
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            if (__any_sync(0xffffffffu, at > queue + 2048 * (SR_QUEUE - 8))) drain();
#pragma unroll
            for (int j = 8 * g; j < 8 * g + 8; ++j) sc_push(at, x(j), cx[KC - 1], id + j);
          }
        }
      };
#pragma unroll 1
      for (int c = 0; c < cols; c += 64) {
        take(c, 0);
        take(c + 32, 32);
#pragma unroll
        for (int j = 0; j < 64; ++j) z[j] = z[j + 64];   // the other half to the front
      }
    }
    drain();
    if (row < a.n) {
      const size_t at = (size_t)row * a.slices + 2 * group + half;
      a.rec.stat[at] = make_float4(m, l, sx, 0.f);
#pragma unroll
      for (int p = 0; p < KC; ++p) {
        a.rec.top_x[((size_t)row * KC + p) * a.slices + 2 * group + half] = cx[p] * rs;
        a.rec.top_v[((size_t)row * KC + p) * a.slices + 2 * group + half] = cv[p];
      }
    }
    __syncwarp();
  }
  __syncthreads();
  sc_settle(bars, a.stages, a.flag);
  if (warp == 9) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

// Vocabulary-major variant for few rows: bn <= 128 vocabulary entries are the
// MMA's M side, the rows' hi and lo parts (tp each, a multiple of 8) its N side, so
// the matrix work follows the number of rows and the kernel streams the
// embedding once.  The epilogue adds the two parts, transposes the logits
// through shared memory and gives each row to a warp.
constexpr int SV_THREADS = 320;
constexpr int SV_MAX_ROWS = 56;
constexpr int SV_KBS = 2;          // k blocks per stage

template <int KC>
__global__ void __launch_bounds__(SV_THREADS, 1)
    score_vocab_kernel(const __grid_constant__ CUtensorMap map_y, const __grid_constant__ CUtensorMap map_e, ScoreTc a) {
  extern __shared__ uint8_t sv_raw[];
  __shared__ ScoreBars bars;
  __shared__ float st[SV_MAX_ROWS][3];
  __shared__ float lx[SV_MAX_ROWS][KC];
  __shared__ int lv[SV_MAX_ROWS][KC];
  __shared__ float ex[8][32];                       // a warp's entrants
  __shared__ int ev[8][32];
  uint8_t* smem = (uint8_t*)(((uintptr_t)sv_raw + 1023) & ~(uintptr_t)1023);
  constexpr int ZLD = 132;
  float* zb = reinterpret_cast<float*>(smem + (size_t)a.stages * a.stage_bytes);   // [tp][ZLD]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tp = a.pad;
  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(&bars.full[s], 1);
      mbar_init(&bars.empty[s], 1);
    }
    for (int s = 0; s < a.slots; ++s) {
      mbar_init(&bars.acc_full[s], 1);
      mbar_init(&bars.acc_empty[s], 4);
    }
    mbar_init(&bars.drained, 1);
    bars.abort = bars.issued = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncwarp();
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&bars.tmem)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  for (int i = threadIdx.x; i < SV_MAX_ROWS; i += SV_THREADS) {
    st[i][0] = -INFINITY;
    st[i][1] = st[i][2] = 0.f;
    for (int p = 0; p < KC; ++p) {
      lx[i][p] = -INFINITY;
      lv[i][p] = 0x7fffffff;
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = bars.tmem;
  const uint32_t ybytes = (uint32_t)(2 * tp) * 128, ebytes = (uint32_t)a.bn * 128;
  const uint32_t slot_cols = (uint32_t)(2 * tp + 31) & ~31u;

  // A stage holds up to two k blocks: their embedding rows (16 KB each), then their
  // activations.
  const uint32_t ybase = SV_KBS * 16384, ystep = (ybytes + 1023) & ~1023u;
  const int spt = (a.nkb + SV_KBS - 1) / SV_KBS;       // stages per tile
  if (warp == 8) {
    if (lane == 0) {
      const int total = min(a.copies, (a.vt - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x * spt);
      const int v_step = (int)gridDim.x * a.bn;
      auto copy_e = [&](int s, int k0, int v0) {     // expect the stage, request its embedding rows
        uint8_t* sp = smem + (size_t)s * a.stage_bytes;
        const bool two = k0 + 1 < a.nkb;
        sc_expect(&bars.full[s], two ? 2 * (ybytes + ebytes) : ybytes + ebytes);
        sc_copy(&bars.full[s], sp, &map_e, k0 * SC_BK, v0);
        if (two) sc_copy(&bars.full[s], sp + 16384, &map_e, (k0 + 1) * SC_BK, v0);
      };
      // the embedding of the first stages is requested before the wait for pass 0:
      // pass 0 has itself waited for everything before it
      const int ahead = min(a.stages, total);
      int k0 = 0, v0 = (int)blockIdx.x * a.bn;
      for (int i = 0; i < ahead; ++i) {
        copy_e(i, k0, v0);
        if ((k0 += SV_KBS) >= a.nkb) {
          k0 = 0;
          v0 += v_step;
        }
      }
      pdl_enter();
      int s = 0, ph = 1, issued = 0, ky = 0;
      for (; issued < total; ++issued) {
        if (issued >= a.stages) {
          if (!sc_wait(&bars.empty[s], ph, &bars.abort, a.wait_ns)) {
            atomicExch(&bars.abort, 1);
            break;
          }
          copy_e(s, k0, v0);
          if ((k0 += SV_KBS) >= a.nkb) {
            k0 = 0;
            v0 += v_step;
          }
        }
        uint8_t* sp = smem + (size_t)s * a.stage_bytes + ybase;
        sc_copy(&bars.full[s], sp, &map_y, ky * SC_BK, 0);
        if (ky + 1 < a.nkb) sc_copy(&bars.full[s], sp + ystep, &map_y, (ky + 1) * SC_BK, 0);
        if ((ky += SV_KBS) >= a.nkb) ky = 0;
        if (++s == a.stages) {
          s = 0;
          ph ^= 1;
        }
      }
      bars.issued = issued;
    }
    __syncwarp();
  } else if (warp == 9) {
    if (lane == 0) {
      pdl_enter();
      const uint32_t idesc = (1u << 4) | ((uint32_t)(2 * tp >> 3) << 17) | (8u << 24);
      const uint64_t desc0 = smem_desc_sw128(smem_u32(smem));
      int s = 0, ph = 0, slot = 0, slot_ph = 1, used = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < a.vt && ok; t += gridDim.x) {
        for (int c0 = 0; c0 < a.nkb && ok; c0 += SC_CHUNK) {
          if (used >= a.slots) ok = sc_wait(&bars.acc_empty[slot], slot_ph, &bars.abort, a.wait_ns);
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint32_t acc = tmem + slot * slot_cols;
          for (int k0 = c0; k0 < min(c0 + SC_CHUNK, a.nkb) && ok; k0 += SV_KBS) {
            ok = sc_wait(&bars.full[s], ph, &bars.abort, a.wait_ns);
            if (!ok) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint64_t e0 = desc0 + (uint64_t)(s * (a.stage_bytes >> 4)), y0 = e0 + (ybase >> 4);
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) sc_mma(acc, e0 + 2 * ks, y0 + 2 * ks, idesc, k0 != c0 || ks != 0);
            if (k0 + 1 < a.nkb) {
              const uint64_t e1 = e0 + (16384 >> 4), y1 = y0 + (ystep >> 4);
#pragma unroll
              for (int ks = 0; ks < 4; ++ks) sc_mma(acc, e1 + 2 * ks, y1 + 2 * ks, idesc, true);
            }
            sc_commit(&bars.empty[s]);
            if (++s == a.stages) {
              s = 0;
              ph ^= 1;
            }
          }
          if (ok) sc_commit(&bars.acc_full[slot]);
          ++used;
          if (++slot == a.slots) {
            slot = 0;
            slot_ph ^= 1;
          }
        }
      }
      if (!ok) atomicExch(&bars.abort, 1);
    }
    __syncwarp();
  } else {
    pdl_enter();
    const uint32_t laddr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    bool ok = true;
    int slot = 0, slot_ph = 0;
    for (int t = blockIdx.x; t < a.vt; t += gridDim.x) {
      if (warp < 4) {
        float z[64];                                     // an entry's logits
        for (int c0 = 0; c0 < a.nkb; c0 += SC_CHUNK) {
          ok = warp_wait(&bars.acc_full[slot], slot_ph, &bars.abort, true, a.wait_ns);
          if (!ok) break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll
          for (int c = 0; c < 64; c += 16) {
            if (c >= tp) continue;
            // hi and lo of 16 rows; the last eight may be the next part's or none's, not used
            uint32_t hi[16], lo[16];
            sc_ld16(hi, laddr + slot * slot_cols + c);
            sc_ld16(lo, laddr + slot * slot_cols + c + tp);
            sc_ld_wait(hi);
            sc_pin16(lo);
#pragma unroll
            for (int q = 0; q < 16; ++q) {
              const float x = __uint_as_float(hi[q]) + __uint_as_float(lo[q]);
              z[c + q] = c0 == 0 ? x : z[c + q] + x;
            }
          }
          asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.acc_empty[slot]);
          if (++slot == a.slots) {
            slot = 0;
            slot_ph ^= 1;
          }
        }
        if (ok) {
#pragma unroll
          for (int c = 0; c < SV_MAX_ROWS; ++c)
            if (c < tp) zb[c * ZLD + warp * 32 + lane] = z[c];
        } else if (lane == 0) {
          atomicExch(&bars.abort, 1);
        }
      }
      if (sc_barrier_or(!ok)) break;
      const int v0 = t * a.bn, valid = min(a.bn, a.V - v0);
      for (int row = warp; row < a.n; row += 8) {
        const float rs = a.scale[row], rs2 = rs * kLog2e;
        float x[4], top = -INFINITY;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int i = lane + 32 * q;
          x[q] = i < valid ? zb[row * ZLD + i] : -INFINITY;
          top = fmaxf(top, x[q]);
        }
        float tmax = top;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) tmax = fmaxf(tmax, __shfl_xor_sync(0xffffffffu, tmax, o));
        const float m_old = st[row][0], m = fmaxf(m_old, tmax * rs2);
        float l = 0.f, sx = 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (lane + 32 * q < valid) {
            const float tt = fmaf(x[q], rs2, -m), e = sc_ex2(tt);
            l += e;
            sx = fmaf(e, tt, sx);
          }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          l += __shfl_xor_sync(0xffffffffu, l, o);
          sx += __shfl_xor_sync(0xffffffffu, sx, o);
        }
        const float l_old = st[row][1], s_old = st[row][2];
        __syncwarp();
        if (lane == 0) {
          if (l_old != 0.f) {
            const float dm = m_old - m, f = sc_ex2(dm);
            sx += (s_old + l_old * dm) * f;
            l += l_old * f;
          }
          st[row][0] = m;
          st[row][1] = l;
          st[row][2] = sx;
        }
        // Entrants of the row's list.  More than a warp's worth of them (a first
        // tile) are cut at the kc-th best of the lanes' own best, a bound of the
        // tile's kc-th best from below.
        const float worst = lx[row][KC - 1];
        float cut = worst;
        int hits = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) hits += __popc(__ballot_sync(0xffffffffu, x[q] > worst));
        if (hits > 32) {
          int rank = 0;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float o = __shfl_sync(0xffffffffu, top, j);
            rank += o > top || (o == top && j < lane);
          }
          // just below the lane's best of that rank, so that the test stays x > cut
          const float kth = __shfl_sync(0xffffffffu, top, __ffs(__ballot_sync(0xffffffffu, rank == KC - 1)) - 1);
          cut = fmaxf(worst, sc_below(kth));
          hits = 0;
#pragma unroll
          for (int q = 0; q < 4; ++q) hits += __popc(__ballot_sync(0xffffffffu, x[q] > cut));
        }
        // in rounds of 32 at most (one, but for many equal logits): the entrants to
        // lanes, then every entry's place by counting who is before it
        int done = 0;
        while (done < hits) {
          int before = 0;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const unsigned m4 = __ballot_sync(0xffffffffu, x[q] > cut);
            const int at = before + __popc(m4 & ((1u << lane) - 1)) - done;
            if (x[q] > cut && at >= 0 && at < 32) {
              ex[warp][at] = x[q];
              ev[warp][at] = v0 + lane + 32 * q;
            }
            before += __popc(m4);
          }
          const int cnt = min(32, hits - done);
          done += 32;
          __syncwarp();
          const float nx = lane < cnt ? ex[warp][lane] : -INFINITY, ox = lane < KC ? lx[row][lane] : -INFINITY;
          const int nv = lane < cnt ? ev[warp][lane] : 0x7fffffff, ov = lane < KC ? lv[row][lane] : 0x7fffffff;
          int nr = 0, orank = lane;                    // the list is sorted
          for (int i = 0; i < KC; ++i) nr += sc_better(lx[row][i], lv[row][i], nx, nv);
          for (int i = 0; i < cnt; ++i) {
            const float ix = ex[warp][i];
            const int iv = ev[warp][i];
            nr += sc_better(ix, iv, nx, nv);
            orank += sc_better(ix, iv, ox, ov);
          }
          __syncwarp();
          if (lane < KC && orank < KC) {
            lx[row][orank] = ox;
            lv[row][orank] = ov;
          }
          if (lane < cnt && nr < KC) {
            lx[row][nr] = nx;
            lv[row][nr] = nv;
          }
          __syncwarp();
        }
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");   // zb is free again
    }
    __syncwarp();
    for (int row = warp; row < a.n; row += 8) {
      const size_t at = (size_t)row * a.slices + blockIdx.x;
      if (lane == 0) a.rec.stat[at] = make_float4(st[row][0], st[row][1], st[row][2], 0.f);
      if (lane < KC) {
        a.rec.top_x[((size_t)row * KC + lane) * a.slices + blockIdx.x] = lx[row][lane] * a.scale[row];
        a.rec.top_v[((size_t)row * KC + lane) * a.slices + blockIdx.x] = lv[row][lane];
      }
    }
  }
  __syncthreads();
  sc_settle(bars, a.stages, a.flag);
  if (warp == 9) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

// ------------------------------------------------------------------ pass 2
constexpr int SM_THREADS = 256, SM_WARPS = SM_THREADS / 32;
constexpr int kMaxSlices = 2 * kScoreSms;
constexpr int SM_PER = (kMaxSlices + SM_THREADS - 1) / SM_THREADS;   // lists of a thread

struct ScoreCand {
  float x;
  int v;
};

// One warp: the outputs of a row with a logit that is not finite.
__device__ __forceinline__ void score_not_finite(const ScoreArgs& a, int row, int target) {
  const int lane = threadIdx.x & 31;
  if (lane == 0 && a.entropy) a.entropy[row] = CUDART_NAN_F;
  if (lane == 0 && a.logp) a.logp[row] = target < 0 ? 0.f : CUDART_NAN_F;
  if (lane < a.k) {
    a.top_ids[(size_t)row * a.k + lane] = -1;
    a.top_logp[(size_t)row * a.k + lane] = CUDART_NAN_F;
  }
}

// One warp: a row's outputs from its statistics, its chosen tokens (ids, logits by pass 1
// in `fast`, by fp64 in zs) and the given token's logit zs[n_pick].  Where a few tokens
// have most of the probability, the errors of their pass 1 logits are what the sums are
// off by: the chosen tokens' terms are replaced by those of their fp64 logits.
__device__ __forceinline__ void score_finish(const ScoreArgs& a, int row, float M, float L, float S, int n_pick,
                                             int target, const double* zs, const int* ids, const float* fast) {
  constexpr double kLn2 = 0.693147180559945309;
  const int lane = threadIdx.x & 31;
  double dl = 0.0, ds = 0.0;
  if (lane < n_pick) {
    // t0 as pass 1 had it.  e^t1 - e^t0 from the difference: both corrections need few bits
    const double t1 = zs[lane] / kLn2 - (double)M, t0 = (double)fast[lane] * (double)kLog2e - (double)M;
    const float e0 = exp2f((float)t0), step = (float)((t1 - t0) * kLn2);
    dl = (double)e0 * (double)expm1f(step);
    ds = dl * t1 + (double)e0 * (t1 - t0);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    dl += __shfl_xor_sync(0xffffffffu, dl, o);
    ds += __shfl_xor_sync(0xffffffffu, ds, o);
  }
  const double l = (double)L + dl, log_l = log(l), lse = (double)M * kLn2 + log_l;
  if (lane == 0 && a.entropy) a.entropy[row] = (float)(log_l - ((double)S + ds) / l * kLn2);
  if (lane == 0 && a.logp)
    a.logp[row] = target < 0 ? 0.f : target >= a.V ? CUDART_NAN_F : (float)(zs[n_pick] - lse);
  // the chosen ones' final order
  if (lane < n_pick) {
    const double z = zs[lane];
    const int id = ids[lane];
    int rank = 0;
    for (int i = 0; i < n_pick; ++i) rank += zs[i] > z || (zs[i] == z && ids[i] < id);
    if (rank < a.k) {
      a.top_ids[(size_t)row * a.k + rank] = id;
      a.top_logp[(size_t)row * a.k + rank] = (float)(z - lse);
    }
  }
}

// One CTA per row.  The kc-th best of 32 groups' best list heads bounds the kc-th
// best logit from below, so only entries at or above it are candidates: a few
// more than kc, whatever the number of lists.  They are ranked by counting; the
// chosen and the given token are scored in fp64, two tokens a warp.  With one CTA
// on the SM every step is a round trip: loads that do not depend on one another
// are issued together.  (128 threads, twice the CTAs per SM, took 25 us longer over
// 1024 rows.)
__global__ void __launch_bounds__(SM_THREADS, 3) score_merge_kernel(ScoreArgs a, int kc, ScoreTc tc) {
  pdl_enter();
  extern __shared__ double sm_dyn[];
  double* yd = sm_dyn;                                              // [d] the row's activations
  ScoreCand* cand = reinterpret_cast<ScoreCand*>(sm_dyn + a.d);     // [slices * kc]
  __shared__ float wred[3][SM_WARPS];
  __shared__ float gmax[SM_WARPS][32];
  __shared__ float bound;
  __shared__ int n_cand;
  __shared__ double zs[kMaxCand + 1];
  __shared__ int ids[kMaxCand + 1];
  __shared__ float fast[kMaxCand];          // the chosen ones' logits by pass 1
  const int row = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slices = tc.slices;
  const float4* stat = tc.rec.stat + (size_t)row * slices;
  const float* gx = tc.rec.top_x + (size_t)row * kc * slices;
  const int* gv = tc.rec.top_v + (size_t)row * kc * slices;
  const float* yr = a.y + (size_t)row * a.y_stride;
  const int target = a.targets ? a.targets[row] : -1;
  const int gave_up = *tc.flag;
  float4 v[SM_PER];
  float hx[SM_PER];
#pragma unroll
  for (int u = 0; u < SM_PER; ++u) {
    const int i = tid + u * SM_THREADS;
    v[u] = i < slices ? stat[i] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
    hx[u] = i < slices ? gx[i] : -INFINITY;
  }
  for (int j = 4 * tid; j < a.d; j += 4 * SM_THREADS) {
    const float4 f = *reinterpret_cast<const float4*>(yr + j);
    *reinterpret_cast<double2*>(yd + j) = make_double2((double)f.x, (double)f.y);
    *reinterpret_cast<double2*>(yd + j + 2) = make_double2((double)f.z, (double)f.w);
  }
  // statistics, in a fixed order: a thread's slices, lanes, warps
  float M = -INFINITY, head = -INFINITY;
  bool bad = gave_up != 0;
#pragma unroll
  for (int u = 0; u < SM_PER; ++u) {
    bad |= isnan(v[u].y) || isnan(v[u].z);
    M = fmaxf(M, v[u].x);
    head = fmaxf(head, hx[u]);
  }
  gmax[warp][lane] = head;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (lane == 0) wred[0][warp] = M;
  if (tid == 0) n_cand = 0;
  bad = __syncthreads_or(bad);
  if (warp == 0) {
    float g = gmax[0][lane];
#pragma unroll
    for (int w = 1; w < SM_WARPS; ++w) g = fmaxf(g, gmax[w][lane]);
    int rank = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const float o = __shfl_sync(0xffffffffu, g, j);
      rank += o > g || (o == g && j < lane);
    }
    if (rank == kc - 1) bound = g;
  }
#pragma unroll
  for (int w = 0; w < SM_WARPS; ++w) M = fmaxf(M, wred[0][w]);
  float L = 0.f, S = 0.f;
#pragma unroll
  for (int u = 0; u < SM_PER; ++u) {
    if (v[u].x == -INFINITY) continue;
    const float dm = v[u].x - M, f = exp2f(dm);
    L += v[u].y * f;
    S += (v[u].z + v[u].y * dm) * f;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    L += __shfl_xor_sync(0xffffffffu, L, o);
    S += __shfl_xor_sync(0xffffffffu, S, o);
  }
  if (lane == 0) {
    wred[1][warp] = L;
    wred[2][warp] = S;
  }
  __syncthreads();
  L = S = 0.f;
#pragma unroll
  for (int w = 0; w < SM_WARPS; ++w) {
    L += wred[1][w];
    S += wred[2][w];
  }
  bad = bad || !isfinite(M) || !isfinite(L);
  if (bad) {
    if (warp == 0) score_not_finite(a, row, target);
    return;
  }
  // candidates: a list's entries from its head down to the bound, four at a time
#pragma unroll
  for (int u = 0; u < SM_PER; ++u) {
    const int i = tid + u * SM_THREADS;
    if (i >= slices || !(hx[u] >= bound)) continue;
    bool more = true;
    for (int p0 = 0; p0 < kc && more; p0 += 4) {      // kc is a multiple of 4
      float x4[4];
      int v4[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        x4[q] = gx[(size_t)(p0 + q) * slices + i];
        v4[q] = gv[(size_t)(p0 + q) * slices + i];
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        more = more && x4[q] >= bound && v4[q] != 0x7fffffff;
        if (more) {
          const int at = atomicAdd(&n_cand, 1);
          cand[at].x = x4[q];
          cand[at].v = v4[q];
        }
      }
    }
  }
  const int n_pick = min(max(a.k, kSpare) + kSpare, a.V);
  if (tid == 0) ids[n_pick] = target;
  __syncthreads();
  // a candidate's rank: how many come before it (their order in memory is of no matter)
  const int nc = n_cand;
  for (int i = warp; i < nc; i += SM_WARPS) {
    const float x = cand[i].x;
    const int id = cand[i].v;
    int rank = 0;
    for (int j = lane; j < nc; j += 32) rank += sc_better(cand[j].x, cand[j].v, x, id);
    rank = __reduce_add_sync(0xffffffffu, rank);
    if (lane == 0 && rank < n_pick) {
      ids[rank] = id;
      fast[rank] = x;
    }
  }
  __syncthreads();
  for (int p0 = warp; p0 <= n_pick; p0 += 2 * SM_WARPS) {
    // two tokens, 1024 elements of each requested at once
    double acc[2][2] = {{0.0, 0.0}, {0.0, 0.0}};
    const __half* e[2];
    bool has[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int p = p0 + u * SM_WARPS, id = p <= n_pick ? ids[p] : -1;
      has[u] = id >= 0 && id < a.V;
      e[u] = a.E + (size_t)(has[u] ? id : 0) * a.d;
    }
    for (int j0 = 8 * lane; j0 < a.d; j0 += 1024) {
      uint4 w[2][4];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          w[u][q] = has[u] && j0 + 256 * q < a.d ? *reinterpret_cast<const uint4*>(e[u] + j0 + 256 * q)
                                                 : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (j0 + 256 * q >= a.d) break;
        double2 yy[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) yy[i] = *reinterpret_cast<const double2*>(yd + j0 + 256 * q + 2 * i);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (!has[u]) continue;
          const uint32_t ww[4] = {w[u][q].x, w[u][q].y, w[u][q].z, w[u][q].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&ww[i]));
            acc[u][0] = fma((double)f.x, yy[i].x, acc[u][0]);
            acc[u][1] = fma((double)f.y, yy[i].y, acc[u][1]);
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      double z = acc[u][0] + acc[u][1];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
      if (lane == 0 && p0 + u * SM_WARPS <= n_pick) zs[p0 + u * SM_WARPS] = z;
    }
  }
  __syncthreads();
  if (warp == 0) score_finish(a, row, M, L, S, n_pick, target, zs, ids, fast);
}

// The same with a warp per row, for more rows than the CTA form has places for at once
// (three per SM): the steps are round trips and fp64 products, so what counts is how
// many rows are on their way together.  These rows have few lists (kWarpSlices at most).
// Vocabulary 50257, d 2048, k 3, us by CTAs and by warps: 400 rows 14 and 18, 512 rows 23
// and 18, 1021 rows 34 and 18, 4096 rows 111 and 51.
constexpr int SW_WARPS = 4;
constexpr int kMergeRows = 3 * kScoreSms;
constexpr int kWarpSlices = 2 * (kScoreSms / ((kMergeRows + 127) / 128));
constexpr int SW_PER = (kWarpSlices + 31) / 32;   // lists of a lane
constexpr int SW_TOKENS = 6;                      // tokens scored together
constexpr int SW_K = 1024;                        // elements of each on the way at once
constexpr int SW_BYTES = SW_K * (4 + 2 * SW_TOKENS);   // a warp's shared memory: candidates, then these
static_assert(kWarpSlices * kMaxCand * sizeof(ScoreCand) <= SW_BYTES, "a row's candidates fit");

__device__ __forceinline__ void sc_copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

__global__ void __launch_bounds__(32 * SW_WARPS) score_merge_rows_kernel(ScoreArgs a, int kc, ScoreTc tc) {
  pdl_enter();
  extern __shared__ double sm_dyn[];
  __shared__ double all_zs[SW_WARPS][kMaxCand + 1];
  __shared__ int all_ids[SW_WARPS][kMaxCand + 1];
  __shared__ float all_fast[SW_WARPS][kMaxCand];
  __shared__ int counts[SW_WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = blockIdx.x * SW_WARPS + warp;
  if (row >= a.n) return;
  const int slices = tc.slices;
  char* mine = reinterpret_cast<char*>(sm_dyn) + warp * SW_BYTES;
  ScoreCand* cand = reinterpret_cast<ScoreCand*>(mine);
  float* ybuf = reinterpret_cast<float*>(mine);
  __half* ebuf = reinterpret_cast<__half*>(ybuf + SW_K);
  double* zs = all_zs[warp];
  int* ids = all_ids[warp];
  float* fast = all_fast[warp];
  const float4* stat = tc.rec.stat + (size_t)row * slices;
  const float* gx = tc.rec.top_x + (size_t)row * kc * slices;
  const int* gv = tc.rec.top_v + (size_t)row * kc * slices;
  const float* yr = a.y + (size_t)row * a.y_stride;
  const int target = a.targets ? a.targets[row] : -1;
  bool bad = *tc.flag != 0;
  float4 v[SW_PER];
  float hx[SW_PER];
  if (lane == 0) counts[warp] = 0;
#pragma unroll
  for (int u = 0; u < SW_PER; ++u) {
    const int i = lane + 32 * u;
    v[u] = i < slices ? stat[i] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
    hx[u] = i < slices ? gx[i] : -INFINITY;
  }
  // statistics, in a fixed order: a lane's slices, lanes
  float M = -INFINITY, head = -INFINITY;
#pragma unroll
  for (int u = 0; u < SW_PER; ++u) {
    bad |= isnan(v[u].y) || isnan(v[u].z);
    M = fmaxf(M, v[u].x);
    head = fmaxf(head, hx[u]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float L = 0.f, S = 0.f;
#pragma unroll
  for (int u = 0; u < SW_PER; ++u) {
    if (v[u].x == -INFINITY) continue;
    const float dm = v[u].x - M, f = exp2f(dm);
    L += v[u].y * f;
    S += (v[u].z + v[u].y * dm) * f;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    L += __shfl_xor_sync(0xffffffffu, L, o);
    S += __shfl_xor_sync(0xffffffffu, S, o);
  }
  if (__any_sync(0xffffffffu, bad) || !isfinite(M) || !isfinite(L)) {
    score_not_finite(a, row, target);
    return;
  }
  int head_rank = 0;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    const float o = __shfl_sync(0xffffffffu, head, j);
    head_rank += o > head || (o == head && j < lane);
  }
  const float bound =
      __shfl_sync(0xffffffffu, head, __ffs(__ballot_sync(0xffffffffu, head_rank == kc - 1)) - 1);
  // candidates: a list's entries from its head down to the bound, four at a time
#pragma unroll
  for (int u = 0; u < SW_PER; ++u) {
    const int i = lane + 32 * u;
    if (i >= slices || !(hx[u] >= bound)) continue;
    bool more = true;
    for (int p0 = 0; p0 < kc && more; p0 += 4) {      // kc is a multiple of 4
      float x4[4];
      int v4[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        x4[q] = gx[(size_t)(p0 + q) * slices + i];
        v4[q] = gv[(size_t)(p0 + q) * slices + i];
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        more = more && x4[q] >= bound && v4[q] != 0x7fffffff;
        if (more) {
          const int at = atomicAdd(&counts[warp], 1);
          cand[at].x = x4[q];
          cand[at].v = v4[q];
        }
      }
    }
  }
  const int n_pick = min(max(a.k, kSpare) + kSpare, a.V);
  if (lane == 0) ids[n_pick] = target;
  __syncwarp();
  // a candidate's rank: how many come before it (their order in memory is of no matter)
  const int nc = *(volatile int*)&counts[warp];
  for (int i = lane; i < nc; i += 32) {
    const ScoreCand me = cand[i];
    int rank = 0;
    for (int j = 0; j < nc; ++j) rank += sc_better(cand[j].x, cand[j].v, me.x, me.v);
    if (rank < n_pick) {
      ids[rank] = me.v;
      fast[rank] = me.x;
    }
  }
  __syncwarp();
  // fp64 products: SW_K elements of y and of SW_TOKENS tokens requested at once; a lane
  // reads what it copied
  for (int p0 = 0; p0 <= n_pick; p0 += SW_TOKENS) {
    double acc[SW_TOKENS];
    const __half* e[SW_TOKENS];
#pragma unroll
    for (int u = 0; u < SW_TOKENS; ++u) {
      const int id = p0 + u <= n_pick ? ids[p0 + u] : -1;
      acc[u] = 0.0;
      e[u] = id >= 0 && id < a.V ? a.E + (size_t)id * a.d : nullptr;
    }
    for (int d0 = 0; d0 < a.d; d0 += SW_K) {
      const int nd = min(SW_K, a.d - d0);
      for (int j = 8 * lane; j < nd; j += 256) {
        sc_copy16(ybuf + j, yr + d0 + j);
        sc_copy16(ybuf + j + 4, yr + d0 + j + 4);
#pragma unroll
        for (int u = 0; u < SW_TOKENS; ++u)
          if (e[u]) sc_copy16(ebuf + u * SW_K + j, e[u] + d0 + j);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      for (int j = 8 * lane; j < nd; j += 256) {
        const float4 y0 = *reinterpret_cast<const float4*>(ybuf + j), y1 = *reinterpret_cast<const float4*>(ybuf + j + 4);
        const double yy[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
#pragma unroll
        for (int u = 0; u < SW_TOKENS; ++u) {
          if (!e[u]) continue;
          const uint4 w = *reinterpret_cast<const uint4*>(ebuf + u * SW_K + j);
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&ww[i]));
            acc[u] = fma((double)f.x, yy[2 * i], acc[u]);
            acc[u] = fma((double)f.y, yy[2 * i + 1], acc[u]);
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < SW_TOKENS; ++u) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[u] += __shfl_xor_sync(0xffffffffu, acc[u], o);
      if (lane == 0 && p0 + u <= n_pick) zs[p0 + u] = acc[u];
    }
  }
  __syncwarp();
  score_finish(a, row, M, L, S, n_pick, target, zs, ids, fast);
}

size_t score_merge_smem(int slices, int kc, int d) { return (size_t)d * 8 + (size_t)slices * kc * sizeof(ScoreCand); }

// candidates a slice keeps: k + kSpare (at least 2 kSpare, for the sum's sake), in the
// sizes that are instantiated
int score_cand(int k) { return k + kSpare <= 4 ? 4 : k + kSpare <= 8 ? 8 : k + kSpare <= 12 ? 12 : 20; }

constexpr int kScoreChunk = 37 * 128;  // rows per sweep over the embedding: bounds the workspace; 37 row
                                       // tiles share 148 SMs evenly
constexpr size_t kVocabSmem = 213 * 1024;   // beside up to 13 KB of static shared memory
constexpr size_t kRowsSmem = 226 * 1024;

struct ScorePlan {
  ScoreTc t;
  bool by_rows;
  int grid;
  size_t smem, parts_off, scale_off, stat_off, top_x_off, top_v_off, bytes;
};

// Up to 56 rows the embedding streams as the M side (its bytes are the bound); above,
// the rows are (the matrix work is).  Vocabulary 50257, d 2048, k 5, vocabulary-major
// and row-major:  8 rows 51 and 66 us, 32 rows 55 and 68, 48 rows 63 and 69, 56 rows 68
// and 70, 64 rows 73 and 71 (128 rows row-major 74).
ScorePlan score_plan(int n, int V, int d, int k) {
  ScorePlan p;
  memset(&p, 0, sizeof(p));
  ScoreTc& t = p.t;
  t.n = n;
  t.V = V;
  t.nkb = d / SC_BK;
  p.by_rows = n > SV_MAX_ROWS;
  if (!p.by_rows) {
    t.pad = (n + 7) / 8 * 8;
    // equal tiles: every CTA the same number of them, none above 128 entries
    const int per = (V + kScoreSms - 1) / kScoreSms, tiles = (per + 127) / 128;
    t.bn = std::max(8, (per + tiles - 1) / tiles);
    t.vt = (V + t.bn - 1) / t.bn;
    p.grid = std::min(kScoreSms, t.vt);
    t.slices = p.grid;
    // Two k blocks per stage: a stage costs its copying thread about 0.25 us however
    // small, as long as a k block's rows take from HBM.  One and two blocks: 1 row 49 and
    // 47 us, 32 rows 60 and 56.  At least three stages fit.
    const size_t zb = (size_t)t.pad * 132 * 4;
    t.stage_bytes = SV_KBS * (16384 + (uint32_t)(2 * t.pad * 128 + 1023) / 1024 * 1024);
    t.stages = (int)std::min<size_t>(12, (kVocabSmem - zb - 1024) / t.stage_bytes);
    t.slots = std::min(SC_SLOTS, 512 / ((2 * t.pad + 31) / 32 * 32));
    p.smem = 1024 + (size_t)t.stages * t.stage_bytes + zb;
  } else {
    t.pad = (n + 127) / 128 * 128;
    t.mt = t.pad / 128;
    t.groups = kScoreSms / t.mt;
    // The tile width (a multiple of 32) with the least work on the busiest CTA, counting
    // a tile's fixed cost (its activations' copies, the first k blocks' latency) as 48
    // columns.  Measured at every width: 50257 entries take 128 rows 96 us by 96, 74 by
    // 192, 82 by 256, and 512 rows 207 by 160 and 180 by 256; 2000 entries take 128 rows
    // 36 by 32 and 45 by 256.  The rule is within 7 % of the best width in all of 40
    // combinations of 4 vocabularies, 5 batches and d 512 and 2048, 0.7 % on average.
    long best = -1;
    for (int bn = 256; bn >= 32; bn -= 32) {
      const int vt = (V + bn - 1) / bn;
      const long cost = (long)((vt + t.groups - 1) / t.groups) * (bn + 48);
      if (best < 0 || cost < best) {
        best = cost;
        t.bn = bn;
      }
    }
    t.vt = (V + t.bn - 1) / t.bn;
    t.groups = std::min(t.groups, t.vt);
    p.grid = t.mt * t.groups;
    t.slices = 2 * t.groups;
    t.stage_bytes = 32768 + (uint32_t)t.bn * 128;
    const size_t queue = (size_t)SR_QUEUE * 256 * 8;
    t.stages = (int)std::min<size_t>(12, (kRowsSmem - queue - 1024) / t.stage_bytes);
    p.smem = 1024 + (size_t)t.stages * t.stage_bytes + queue;
  }
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  p.parts_off = 256;               // behind the flag, which has its place whatever the sizes are
  p.scale_off = p.parts_off + up((size_t)2 * t.pad * d * 2);
  p.stat_off = p.scale_off + up((size_t)t.pad * 4);
  p.top_x_off = p.stat_off + up((size_t)n * t.slices * 16);
  const size_t top = up((size_t)n * t.slices * score_cand(k) * 4);
  p.top_v_off = p.top_x_off + top;
  p.bytes = p.top_v_off + top;
  return p;
}

template <int KC>
tl_status launch_score_pass1(const ScorePlan& p, const CUtensorMap& my, const CUtensorMap& me, cudaStream_t s) {
  static std::atomic<uint64_t> attr_done{0};
  TL_TRY(once_per_device(attr_done, []() -> tl_status {
    TL_CUDA(cudaFuncSetAttribute(score_rows_kernel<KC>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRowsSmem));
    TL_CUDA(cudaFuncSetAttribute(score_vocab_kernel<KC>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kVocabSmem));
    // with fewer registers at launch the statistics warpgroups would wait for the rest for good
    cudaFuncAttributes fa;
    TL_CUDA(cudaFuncGetAttributes(&fa, score_rows_kernel<KC>));
    if (fa.numRegs < SR_REGS)
      return set_error(TL_ERR_CUDA, "score_rows_kernel was built with %d registers, not %d", fa.numRegs, SR_REGS);
    return ok();
  }));
  if (p.by_rows) TL_LAUNCH_PDL(score_rows_kernel<KC>, p.grid, SR_THREADS, p.smem, s, my, me, p.t);
  else TL_LAUNCH_PDL(score_vocab_kernel<KC>, p.grid, SV_THREADS, p.smem, s, my, me, p.t);
  return ok();
}

}  // namespace

size_t score_workspace(int n, int V, int d, int k) {
  if (n == 0) return 0;
  size_t b = score_plan(std::min(n, kScoreChunk), V, d, k).bytes;
  if (n > kScoreChunk && n % kScoreChunk) b = std::max(b, score_plan(n % kScoreChunk, V, d, k).bytes);
  return b;
}

tl_status launch_score_head(const ScoreArgs& a0, cudaStream_t s) {
  static std::atomic<uint64_t> attr_done{0};
  TL_TRY(once_per_device(attr_done, []() -> tl_status {
    const int most = (int)score_merge_smem(kMaxSlices, kMaxCand, 8192);
    TL_CUDA(cudaFuncSetAttribute(score_merge_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most));
    TL_CUDA(cudaFuncSetAttribute(score_merge_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 SW_WARPS * SW_BYTES));
    return ok();
  }));
  for (int r0 = 0; r0 < a0.n; r0 += kScoreChunk) {
    ScoreArgs a = a0;
    a.n = std::min(kScoreChunk, a0.n - r0);
    a.y = a0.y + (size_t)r0 * a0.y_stride;
    if (a.targets) a.targets += r0;
    if (a.logp) a.logp += r0;
    if (a.entropy) a.entropy += r0;
    if (a.k) {
      a.top_ids += (size_t)r0 * a.k;
      a.top_logp += (size_t)r0 * a.k;
    }
    ScorePlan p = score_plan(a.n, a.V, a.d, a.k);
    ScoreTc& t = p.t;
    __half* parts = (__half*)(a.ws + p.parts_off);
    float* scale = (float*)(a.ws + p.scale_off);
    t.scale = scale;
    t.flag = (int*)a.ws;
    t.wait_ns = a.wait_ns;
    t.copies = a.copies;
    t.rec.stat = (float4*)(a.ws + p.stat_off);
    t.rec.top_x = (float*)(a.ws + p.top_x_off);
    t.rec.top_v = (int*)(a.ws + p.top_v_off);
    CUtensorMap my, me;
    TL_TRY(encode_2d(&my, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, parts, a.d, 2 * t.pad, (uint64_t)a.d * 2, SC_BK,
                     p.by_rows ? 128 : 2 * t.pad, CU_TENSOR_MAP_SWIZZLE_128B));
    TL_TRY(encode_2d(&me, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, a.E, a.d, a.V, (uint64_t)a.d * 2, SC_BK, t.bn,
                     CU_TENSOR_MAP_SWIZZLE_128B));
    TL_LAUNCH_PDL(score_split_kernel, t.pad, 256, 0, s, a.y, a.y_stride, a.n, a.d, t.pad, parts, scale,
                  r0 == 0 ? t.flag : nullptr);
    const int kc = score_cand(a.k);
    TL_TRY(kc == 4   ? launch_score_pass1<4>(p, my, me, s)
                   : kc == 8 ? launch_score_pass1<8>(p, my, me, s)
                   : kc == 12 ? launch_score_pass1<12>(p, my, me, s) : launch_score_pass1<20>(p, my, me, s));
    if (a.n > kMergeRows)
      TL_LAUNCH_PDL(score_merge_rows_kernel, (a.n + SW_WARPS - 1) / SW_WARPS, 32 * SW_WARPS,
                    (size_t)SW_WARPS * SW_BYTES, s, a, kc, t);
    else
      TL_LAUNCH_PDL(score_merge_kernel, a.n, SM_THREADS, score_merge_smem(t.slices, kc, a.d), s, a, kc, t);
  }
  return ok();
}

}  // namespace tl
