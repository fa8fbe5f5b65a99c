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
// embedding tile on the tensor cores, so a logit has fp32 accuracy for twice the
// matrix work (one fp16 part alone would leave errors of 2^-12 per activation in
// every probability).
// Pass 1 streams the embedding through tcgen05 and keeps, per row and slice of
// the vocabulary, the running maximum m, l = sum e^(z - m), s = sum e^(z - m) (z - m)
// and the best candidates.
// Pass 2, one CTA per row, merges the slices and decides the order of the best
// k + kSpare candidates, and the given token's logit, by fp64 dot products of the
// inputs, so the ranking does not depend on pass 1's rounding (ties go to the
// lowest token id).
#include <math_constants.h>

#include <algorithm>
#include <cstring>

#include "tc_util.cuh"

namespace tl {
namespace {

constexpr int kSpare = 4;          // candidates kept beyond k
constexpr int kMaxCand = 16 + kSpare;
constexpr int SC_BK = 64;          // k per stage (one 128-byte swizzled row)
constexpr int kScoreSms = 148;

__device__ __forceinline__ bool sc_better(float x, int v, float bx, int bv) {
  return x > bx || (x == bx && v < bv);
}

// slice record of one row: m, l, s (base 2, s in units of log2), then kc
// candidates (logit, id), best first
__host__ __device__ inline int rec_words(int kc) { return 3 + 2 * kc; }

__device__ __forceinline__ float sc_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ------------------------------------------------------------------ pass 0
// One CTA per row of the padded batch: parts[row] = hi, parts[pad + row] = lo
// (zeros behind the batch), scale[row] = the power of two taken out.
__global__ void __launch_bounds__(256) score_split_kernel(const float* __restrict__ y, long y_stride, int n, int d,
                                                          int pad, __half* parts, float* scale, int* flag) {
  pdl_enter();
  __shared__ float wmax[8];
  const int row = blockIdx.x, tid = threadIdx.x;
  if (row == 0 && tid == 0) *flag = 0;
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
__device__ __forceinline__ void sc_mma_elect(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n setp.ne.b32 p, %4, 0;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}

// one expect_tx for two copies of the stage, then the copies
__device__ __forceinline__ void sc_expect_elect(uint64_t* bar, uint32_t bytes) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n}\n" ::"r"(smem_u32(bar)),
      "r"(bytes)
      : "memory");
}
__device__ __forceinline__ void sc_copy_elect(uint64_t* bar, void* dst, const CUtensorMap* map, int x, int y) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%1], [%2, "
      "{%3, %4}], [%0];\n}\n" ::"r"(smem_u32(bar)),
      "r"(smem_u32(dst)), "l"(map), "r"(x), "r"(y)
      : "memory");
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
  int units, upc;         // (row tile, vocabulary tile) units, and how many a CTA takes
  int stages;
  uint32_t stage_bytes;
  int slices;             // records per row
  const float* scale;
  float* rec;
  int* flag;              // set when a bounded wait ran out
};

struct ScoreBars {
  uint64_t full[12], empty[12], acc_full[2], acc_empty[2];
  uint32_t tmem;
  int abort;
};

// Row-major variant: 128 rows of activations (hi and lo) are the MMA's M side,
// bn vocabulary entries its N side, so an epilogue thread owns one row and walks
// its logits: the softmax statistics and the candidate list live in registers.
// Warps 0-7 read the accumulators (warp w: TMEM quadrant w mod 4, column half
// w / 4), warp 8 copies, warp 9 issues the MMAs; two accumulators of 256 columns
// let the epilogue of one tile run under the next tile's MMAs.
constexpr int SR_THREADS = 320;

template <int KC>
__global__ void __launch_bounds__(SR_THREADS, 1)
    score_rows_kernel(const __grid_constant__ CUtensorMap map_y, const __grid_constant__ CUtensorMap map_e, ScoreTc a) {
  extern __shared__ uint8_t sr_raw[];
  __shared__ ScoreBars bars;
  uint8_t* smem = (uint8_t*)(((uintptr_t)sr_raw + 1023) & ~(uintptr_t)1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int u0 = blockIdx.x * a.upc, u1 = min(a.units, u0 + a.upc);
  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(&bars.full[s], 1);
      mbar_init(&bars.empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars.acc_full[s], 1);
      mbar_init(&bars.acc_empty[s], 8);
    }
    bars.abort = 0;
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

  if (warp == 8) {
    // ---------------------------------------------------------------- copies
    int s = 0, it = 0, issued = 0;
    bool ok = true;
    for (int u = u0; u < u1 && ok; ++u) {
      const int r0 = u / a.vt * 128, v0 = u % a.vt * a.bn;
      for (int kb = 0; kb < a.nkb; ++kb) {
        if (!warp_wait(&bars.empty[s], (it & 1) ^ 1, &bars.abort, it > 0)) {
          if (lane == 0) atomicExch(&bars.abort, 1);
          ok = false;
          break;
        }
        uint8_t* st = smem + (size_t)s * a.stage_bytes;
        sc_expect_elect(&bars.full[s], a.stage_bytes);
        sc_copy_elect(&bars.full[s], st, &map_y, kb * SC_BK, r0);
        sc_copy_elect(&bars.full[s], st + 16384, &map_y, kb * SC_BK, a.pad + r0);
        sc_copy_elect(&bars.full[s], st + 32768, &map_e, kb * SC_BK, v0);
        ++issued;
        if (++s == a.stages) {
          s = 0;
          ++it;
        }
      }
    }
    if (lane == 0 && *(volatile int*)&bars.abort)      // the copies still in flight land before the CTA leaves
      for (int i = max(0, issued - a.stages); i < issued; ++i) mbar_wait(&bars.full[i % a.stages], (i / a.stages) & 1);
    __syncwarp();
  } else if (warp == 9) {
    // ---------------------------------------------------------------- MMAs
    const uint32_t idesc = (1u << 4) | ((uint32_t)(a.bn >> 3) << 17) | (8u << 24);
    int s = 0, ph = 0;
    bool ok = true;
    for (int u = u0; u < u1 && ok; ++u) {
      const int buf = (u - u0) & 1, use = (u - u0) >> 1;
      ok = warp_wait(&bars.acc_empty[buf], (use & 1) ^ 1, &bars.abort, use > 0);
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t acc = tmem + buf * 256;
      for (int kb = 0; kb < a.nkb && ok; ++kb) {
        ok = warp_wait(&bars.full[s], ph, &bars.abort, true);
        if (!ok) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t st = smem_u32(smem + (size_t)s * a.stage_bytes);
        const uint64_t hi = smem_desc_sw128(st), lo = smem_desc_sw128(st + 16384), e = smem_desc_sw128(st + 32768);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          sc_mma_elect(acc, hi + 2 * ks, e + 2 * ks, idesc, (kb | ks) != 0);
          sc_mma_elect(acc, lo + 2 * ks, e + 2 * ks, idesc, true);
        }
        mma_commit_elect(&bars.empty[s]);
        if (++s == a.stages) {
          s = 0;
          ph ^= 1;
        }
      }
      if (ok) mma_commit_elect(&bars.acc_full[buf]);
    }
    if (!ok && lane == 0) atomicExch(&bars.abort, 1);
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- statistics
    const int half = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t laddr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const int cols = a.bn / 2;                         // a multiple of 16
    float m = -INFINITY, l = 0.f, sx = 0.f;            // in log2 units
    float rs2 = 0.f, rs = 0.f;
    float cx[KC > 0 ? KC : 1];
    int cv[KC > 0 ? KC : 1];
    bool ok = true;
    for (int u = u0; u < u1; ++u) {
      const int mt = u / a.vt, vt = u % a.vt;
      const int row = mt * 128 + r;
      if (u == u0 || vt == 0) {                        // a new row tile
        m = -INFINITY;
        l = sx = 0.f;
        rs = row < a.n ? a.scale[row] : 1.f;
        rs2 = rs * 1.4426950408889634f;
#pragma unroll
        for (int p = 0; p < KC; ++p) {
          cx[p] = -INFINITY;
          cv[p] = 0x7fffffff;
        }
      }
      const int buf = (u - u0) & 1, use = (u - u0) >> 1;
      if (!warp_wait(&bars.acc_full[buf], use & 1, &bars.abort, true)) {
        if (lane == 0) atomicExch(&bars.abort, 1);
        ok = false;
        break;
      }
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const int v0 = vt * a.bn + half * cols;
      const int valid = min(cols, a.V - v0);           // may be <= 0 in the last tile
      uint32_t w[2][16];
      const uint32_t base = laddr + buf * 256 + half * cols;
      sc_ld16(w[0], base);
#pragma unroll 1
      for (int c = 0; c < cols; c += 32) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c0 = c + 16 * h;
          if (c0 >= cols) break;
          sc_ld_wait(w[h]);
          if (c0 + 16 < cols) sc_ld16(w[h ^ 1], base + c0 + 16);
          const int nv = valid - c0;                   // uniform over the warp
          if (nv <= 0) continue;
          float x[16];
          float top = -INFINITY;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            x[j] = __uint_as_float(w[h][j]);
            if (j < nv) top = fmaxf(top, x[j]);
          }
          const float top2 = top * rs2;
          if (top2 > m) {
            const float f = sc_ex2(m - top2);
            sx = l == 0.f ? 0.f : (sx + l * (m - top2)) * f;
            l *= f;
            m = top2;
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            if (j < nv) {
              const float t = fmaf(x[j], rs2, -m), e = sc_ex2(t);
              l += e;
              sx = fmaf(e, t, sx);
            }
          }
          if (KC > 0) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              if (j < nv && x[j] > cx[KC - 1]) {
                // one insertion pass: an equal entry seen earlier (a lower id) stays before
                const float xv = x[j];
                const int id = v0 + c0 + j;
#pragma unroll
                for (int p = KC - 1; p > 0; --p) {
                  const bool up = xv > cx[p - 1], in = xv > cx[p];
                  cv[p] = up ? cv[p - 1] : in ? id : cv[p];
                  cx[p] = up ? cx[p - 1] : in ? xv : cx[p];
                }
                if (xv > cx[0]) {
                  cx[0] = xv;
                  cv[0] = id;
                }
              }
            }
          }
        }
      }
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.acc_empty[buf]);
      if ((u + 1 == u1 || vt + 1 == a.vt) && row < a.n) {
        const int first = mt * a.vt / a.upc;           // the first CTA with units of this row tile
        float* o = a.rec + ((size_t)row * a.slices + 2 * (blockIdx.x - first) + half) * rec_words(KC);
        o[0] = m;
        o[1] = l;
        o[2] = sx;
#pragma unroll
        for (int p = 0; p < KC; ++p) {
          o[3 + 2 * p] = cx[p] * rs;
          o[4 + 2 * p] = __int_as_float(cv[p]);
        }
      }
    }
    if (!ok && lane == 0) atomicExch(a.flag, 1);
    __syncwarp();
  }
  __syncthreads();
  if (warp == 9) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
  if (threadIdx.x == 0 && bars.abort) atomicExch(a.flag, 1);
}

// Vocabulary-major variant for few rows: bn <= 128 vocabulary entries are the
// MMA's M side, the rows' hi and lo parts (tp each, a multiple of 8) its N side, so
// the matrix work follows the number of rows and the kernel streams the
// embedding once.  The epilogue adds the two parts, transposes the logits
// through shared memory and gives each row to a warp.
constexpr int SV_THREADS = 320;
constexpr int SV_MAX_ROWS = 64;

template <int KC>
__global__ void __launch_bounds__(SV_THREADS, 1)
    score_vocab_kernel(const __grid_constant__ CUtensorMap map_y, const __grid_constant__ CUtensorMap map_e, ScoreTc a) {
  extern __shared__ uint8_t sv_raw[];
  __shared__ ScoreBars bars;
  __shared__ float st[SV_MAX_ROWS][3];
  __shared__ float lx[SV_MAX_ROWS][KC > 0 ? KC : 1];
  __shared__ int lv[SV_MAX_ROWS][KC > 0 ? KC : 1];
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
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars.acc_full[s], 1);
      mbar_init(&bars.acc_empty[s], 4);
    }
    bars.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncwarp();
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 256;" ::"r"(smem_u32(&bars.tmem)));
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

  if (warp == 8) {
    // the embedding of the first stages is requested before the wait for pass 0:
    // pass 0 has itself waited for everything before it
    const int total = (a.vt - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x * a.nkb;
    const int ahead = min(a.stages, total);
    int issued = 0;
    bool ok = true;
    for (int i = 0; i < ahead; ++i) {
      uint8_t* sp = smem + (size_t)i * a.stage_bytes;
      sc_expect_elect(&bars.full[i], ybytes + ebytes);
      sc_copy_elect(&bars.full[i], sp, &map_e, i % a.nkb * SC_BK, ((int)blockIdx.x + i / a.nkb * (int)gridDim.x) * a.bn);
    }
    pdl_enter();
    for (int i = 0; i < total && ok; ++i) {
      const int s = i % a.stages, use = i / a.stages;
      const int kb = i % a.nkb, v0 = ((int)blockIdx.x + i / a.nkb * (int)gridDim.x) * a.bn;
      uint8_t* sp = smem + (size_t)s * a.stage_bytes;
      if (use > 0) {
        if (!warp_wait(&bars.empty[s], (use & 1) ^ 1, &bars.abort, true)) {
          if (lane == 0) atomicExch(&bars.abort, 1);
          ok = false;
          break;
        }
        sc_expect_elect(&bars.full[s], ybytes + ebytes);
        sc_copy_elect(&bars.full[s], sp, &map_e, kb * SC_BK, v0);
      }
      sc_copy_elect(&bars.full[s], sp + 16384, &map_y, kb * SC_BK, 0);
      issued = i + 1;
    }
    if (lane == 0 && *(volatile int*)&bars.abort)
      for (int i = max(0, issued - a.stages); i < issued; ++i) mbar_wait(&bars.full[i % a.stages], (i / a.stages) & 1);
    __syncwarp();
  } else if (warp == 9) {
    pdl_enter();
    const uint32_t idesc = (1u << 4) | ((uint32_t)(2 * tp >> 3) << 17) | (8u << 24);
    int s = 0, ph = 0, j = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < a.vt && ok; t += gridDim.x, ++j) {
      const int buf = j & 1, use = j >> 1;
      ok = warp_wait(&bars.acc_empty[buf], (use & 1) ^ 1, &bars.abort, use > 0);
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      for (int kb = 0; kb < a.nkb && ok; ++kb) {
        ok = warp_wait(&bars.full[s], ph, &bars.abort, true);
        if (!ok) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t sp = smem_u32(smem + (size_t)s * a.stage_bytes);
        const uint64_t e = smem_desc_sw128(sp), yy = smem_desc_sw128(sp + 16384);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) sc_mma_elect(tmem + buf * 128, e + 2 * ks, yy + 2 * ks, idesc, (kb | ks) != 0);
        mma_commit_elect(&bars.empty[s]);
        if (++s == a.stages) {
          s = 0;
          ph ^= 1;
        }
      }
      if (ok) mma_commit_elect(&bars.acc_full[buf]);
    }
    if (!ok && lane == 0) atomicExch(&bars.abort, 1);
    __syncwarp();
  } else {
    pdl_enter();
    const uint32_t laddr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    bool ok = true;
    int j = 0;
    for (int t = blockIdx.x; t < a.vt; t += gridDim.x, ++j) {
      const int buf = j & 1, use = j >> 1;
      if (warp < 4) {
        ok = warp_wait(&bars.acc_full[buf], use & 1, &bars.abort, true);
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        if (ok) {
          for (int c = 0; c < tp; c += 8) {
            uint32_t hl[16];                             // hi, then lo
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              uint32_t* d = hl + 8 * q;
              asm volatile(
                  "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                  : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3]), "=r"(d[4]), "=r"(d[5]), "=r"(d[6]), "=r"(d[7])
                  : "r"(laddr + buf * 128 + c + q * tp));
            }
            sc_ld_wait(hl);
#pragma unroll
            for (int q = 0; q < 8; ++q)
              zb[(c + q) * ZLD + warp * 32 + lane] = __uint_as_float(hl[q]) + __uint_as_float(hl[8 + q]);
          }
          asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.acc_empty[buf]);
        } else if (lane == 0) {
          atomicExch(&bars.abort, 1);
        }
      }
      if (sc_barrier_or(!ok)) break;
      const int v0 = t * a.bn, valid = min(a.bn, a.V - v0);
      for (int row = warp; row < a.n; row += 8) {
        const float rs = a.scale[row], rs2 = rs * 1.4426950408889634f;
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
        if (KC > 0) {
          // lane p holds the list's p-th entry
          float cx = lane < KC ? lx[row][lane] : INFINITY;
          int cv = lane < KC ? lv[row][lane] : -1;
          float worst = __shfl_sync(0xffffffffu, cx, KC - 1);
          bool changed = false;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            unsigned hit = __ballot_sync(0xffffffffu, x[q] > worst);   // ids ascend: an equal logit seen later loses
            while (hit) {
              const int src = __ffs(hit) - 1;
              hit &= hit - 1;
              const float xv = __shfl_sync(0xffffffffu, x[q], src);
              if (!(xv > worst)) continue;
              const int id = v0 + src + 32 * q;
              const bool in = xv > cx;
              const float px = __shfl_up_sync(0xffffffffu, cx, 1);
              const int pv = __shfl_up_sync(0xffffffffu, cv, 1);
              const bool up = lane > 0 && xv > px;
              if (lane < KC) {
                cv = up ? pv : in ? id : cv;
                cx = up ? px : in ? xv : cx;
              }
              worst = __shfl_sync(0xffffffffu, cx, KC - 1);
              changed = true;
            }
          }
          if (changed && lane < KC) {
            lx[row][lane] = cx;
            lv[row][lane] = cv;
          }
        }
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");   // zb is free again
    }
    __syncwarp();
    for (int row = warp; row < a.n; row += 8) {
      float* o = a.rec + ((size_t)row * a.slices + blockIdx.x) * rec_words(KC);
      const float rs = a.scale[row];
      if (lane < 3) o[lane] = st[row][lane];
      if (lane < KC) {
        o[3 + 2 * lane] = lx[row][lane] * rs;
        o[4 + 2 * lane] = __int_as_float(lv[row][lane]);
      }
    }
  }
  __syncthreads();
  if (warp == 9) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 256;" ::"r"(tmem));
  }
  if (threadIdx.x == 0 && bars.abort) atomicExch(a.flag, 1);
}

constexpr int SM_THREADS = 256;

// One CTA per row: the slices' statistics and candidates merged, the chosen
// candidates and the given token scored in fp64.
__global__ void __launch_bounds__(SM_THREADS) score_merge_kernel(ScoreArgs a, int kc, ScoreTc tc, int by_rows) {
  pdl_enter();
  __shared__ float wx[SM_THREADS / 32];
  __shared__ int wv[SM_THREADS / 32], wi[SM_THREADS / 32];
  __shared__ double zs[kMaxCand + 1];
  __shared__ int ids[kMaxCand + 1];
  __shared__ float red[2][SM_THREADS / 32];
  const int row = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rw = rec_words(kc);
  const float* base = tc.rec + (size_t)row * tc.slices * rw;
  int slices = tc.slices;
  if (by_rows) {   // the CTAs that had units of this row's tile, two column halves each
    const int mt = row / 128;
    slices = 2 * (((mt + 1) * tc.vt - 1) / tc.upc - mt * tc.vt / tc.upc + 1);
  }
  // statistics, in a fixed order: thread-strided slices, lanes, warps
  float M = -INFINITY;
  bool nan = false;
  for (int i = tid; i < slices; i += SM_THREADS) {
    const float m = base[(size_t)i * rw];
    nan |= isnan(base[(size_t)i * rw + 1]) || isnan(base[(size_t)i * rw + 2]);
    M = fmaxf(M, m);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (lane == 0) wx[warp] = M;
  nan = __syncthreads_or(nan);
  for (int w = 0; w < SM_THREADS / 32; ++w) M = fmaxf(M, wx[w]);
  float L = 0.f, S = 0.f;
  for (int i = tid; i < slices; i += SM_THREADS) {
    const float m = base[(size_t)i * rw];
    if (m == -INFINITY) continue;
    const float dm = m - M, f = exp2f(dm);
    const float l = base[(size_t)i * rw + 1];
    L += l * f;
    S += (base[(size_t)i * rw + 2] + l * dm) * f;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    L += __shfl_xor_sync(0xffffffffu, L, o);
    S += __shfl_xor_sync(0xffffffffu, S, o);
  }
  if (lane == 0) {
    red[0][warp] = L;
    red[1][warp] = S;
  }
  __syncthreads();
  L = S = 0.f;
  for (int w = 0; w < SM_THREADS / 32; ++w) {
    L += red[0][w];
    S += red[1][w];
  }
  const bool bad = nan || !isfinite(M) || !isfinite(L) || *tc.flag != 0;
  constexpr double kLn2 = 0.693147180559945309;
  const double lse = (double)M * kLn2 + log((double)L);
  if (tid == 0 && a.entropy)
    a.entropy[row] = bad ? CUDART_NAN_F : (float)(log((double)L) - (double)S / (double)L * kLn2);

  // candidates: the slices' lists are sorted, so each pick looks at their heads
  int n_pick = bad ? 0 : min(kc, a.V);
  {
    int h0 = 0, h1 = 0;   // heads of this thread's two lists (slices <= 2 * SM_THREADS)
    for (int p = 0; p < n_pick; ++p) {
      float bx = -INFINITY;
      int bv = 0x7fffffff, bi = -1;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int i = tid + u * SM_THREADS, h = u ? h1 : h0;
        if (i < slices && h < kc) {
          const float x = base[(size_t)i * rw + 3 + 2 * h];
          const int v = __float_as_int(base[(size_t)i * rw + 4 + 2 * h]);
          if (sc_better(x, v, bx, bv)) {
            bx = x;
            bv = v;
            bi = i;
          }
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float x = __shfl_xor_sync(0xffffffffu, bx, o);
        const int v = __shfl_xor_sync(0xffffffffu, bv, o), i = __shfl_xor_sync(0xffffffffu, bi, o);
        if (sc_better(x, v, bx, bv)) {
          bx = x;
          bv = v;
          bi = i;
        }
      }
      __syncthreads();
      if (lane == 0) {
        wx[warp] = bx;
        wv[warp] = bv;
        wi[warp] = bi;
      }
      __syncthreads();
      for (int w = 0; w < SM_THREADS / 32; ++w)
        if (sc_better(wx[w], wv[w], bx, bv)) {
          bx = wx[w];
          bv = wv[w];
          bi = wi[w];
        }
      if (bi == tid) ++h0;
      if (bi == tid + SM_THREADS) ++h1;
      if (tid == 0) ids[p] = bv;
    }
  }
  const int target = a.targets ? a.targets[row] : -1;
  if (tid == 0) ids[n_pick] = target;
  __syncthreads();
  for (int p = warp; p <= n_pick; p += SM_THREADS / 32) {
    const int v = ids[p];
    double acc = 0.0;
    if (v >= 0 && v < a.V) {
      const __half* e = a.E + (size_t)v * a.d;
      const float* yr = a.y + (size_t)row * a.y_stride;
      for (int j = 2 * lane; j < a.d; j += 64) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(e + j));
        const float2 yy = *reinterpret_cast<const float2*>(yr + j);
        acc = fma((double)f.y, (double)yy.y, fma((double)f.x, (double)yy.x, acc));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    }
    if (lane == 0) zs[p] = acc;
  }
  __syncthreads();
  if (tid == 0 && a.logp)
    a.logp[row] = target < 0 ? 0.f : target >= a.V || bad ? CUDART_NAN_F : (float)(zs[n_pick] - lse);
  if (tid < a.k && bad) {
    a.top_ids[(size_t)row * a.k + tid] = -1;
    a.top_logp[(size_t)row * a.k + tid] = CUDART_NAN_F;
  }
  // each candidate's rank among them; the first k are the answer
  if (tid < n_pick) {
    int rank = 0;
    for (int p = 0; p < n_pick; ++p) rank += zs[p] > zs[tid] || (zs[p] == zs[tid] && ids[p] < ids[tid]);
    if (rank < a.k) {
      a.top_ids[(size_t)row * a.k + rank] = ids[tid];
      a.top_logp[(size_t)row * a.k + rank] = (float)(zs[tid] - lse);
    }
  }
}

int score_cand(int k) { return k == 0 ? 0 : k <= 4 ? 8 : k <= 8 ? 12 : 20; }

constexpr int kScoreChunk = 4096;      // rows per sweep over the embedding: bounds the workspace
constexpr size_t kScoreSmem = 212 * 1024;   // beside up to 11 KB of static shared memory

struct ScorePlan {
  ScoreTc t;
  bool by_rows;
  int grid;
  size_t smem, parts_off, scale_off, flag_off, rec_off, bytes;
};

// Up to 64 rows the embedding streams as the M side (its bytes are the bound);
// above, the rows are (the matrix work is).
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
    t.stage_bytes = 16384 + (uint32_t)(2 * t.pad * 128 + 1023) / 1024 * 1024;
    const size_t zb = (size_t)t.pad * 132 * 4;
    t.stages = (int)std::min<size_t>(12, (kScoreSmem - zb - 1024) / t.stage_bytes);
    p.smem = 1024 + (size_t)t.stages * t.stage_bytes + zb;
  } else {
    t.pad = (n + 127) / 128 * 128;
    const int mt = t.pad / 128;
    // the tile width (a multiple of 32) with the least work on the busiest CTA,
    // counting a tile's fixed cost as 16 columns
    long best = -1;
    for (int bn = 256; bn >= 128; bn -= 32) {
      const long units = (long)mt * ((V + bn - 1) / bn);
      const long cost = (units + kScoreSms - 1) / kScoreSms * (bn + 16);
      if (best < 0 || cost < best) {
        best = cost;
        t.bn = bn;
      }
    }
    t.vt = (V + t.bn - 1) / t.bn;
    t.units = mt * t.vt;
    t.upc = (t.units + kScoreSms - 1) / kScoreSms;
    p.grid = (t.units + t.upc - 1) / t.upc;
    t.slices = 2 * ((t.vt + t.upc - 1) / t.upc + 1);
    t.stage_bytes = 32768 + (uint32_t)t.bn * 128;
    t.stages = (int)std::min<size_t>(12, (kScoreSmem - 1024) / t.stage_bytes);
    p.smem = 1024 + (size_t)t.stages * t.stage_bytes;
  }
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  p.parts_off = 0;
  p.scale_off = up((size_t)2 * t.pad * d * 2);
  p.flag_off = p.scale_off + up((size_t)t.pad * 4);
  p.rec_off = p.flag_off + 256;
  p.bytes = p.rec_off + up((size_t)n * t.slices * rec_words(score_cand(k)) * 4);
  return p;
}

template <int KC>
tl_status launch_score_pass1(const ScorePlan& p, const CUtensorMap& my, const CUtensorMap& me, cudaStream_t s) {
  static std::atomic<uint64_t> attr_done{0};
  TL_TRY(once_per_device(attr_done, []() -> tl_status {
    TL_CUDA(cudaFuncSetAttribute(score_rows_kernel<KC>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kScoreSmem));
    TL_CUDA(cudaFuncSetAttribute(score_vocab_kernel<KC>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kScoreSmem));
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
    t.flag = (int*)(a.ws + p.flag_off);
    t.rec = (float*)(a.ws + p.rec_off);
    CUtensorMap my, me;
    TL_TRY(encode_2d(&my, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, parts, a.d, 2 * t.pad, (uint64_t)a.d * 2, SC_BK,
                     p.by_rows ? 128 : 2 * t.pad, CU_TENSOR_MAP_SWIZZLE_128B));
    TL_TRY(encode_2d(&me, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, a.E, a.d, a.V, (uint64_t)a.d * 2, SC_BK, t.bn,
                     CU_TENSOR_MAP_SWIZZLE_128B));
    TL_LAUNCH_PDL(score_split_kernel, t.pad, 256, 0, s, a.y, a.y_stride, a.n, a.d, t.pad, parts, scale, t.flag);
    const int kc = score_cand(a.k);
    TL_TRY(kc == 0 ? launch_score_pass1<0>(p, my, me, s)
                   : kc == 8 ? launch_score_pass1<8>(p, my, me, s)
                             : kc == 12 ? launch_score_pass1<12>(p, my, me, s) : launch_score_pass1<20>(p, my, me, s));
    TL_LAUNCH_PDL(score_merge_kernel, a.n, SM_THREADS, 0, s, a, kc, t, p.by_rows ? 1 : 0);
  }
  return ok();
}

}  // namespace tl
