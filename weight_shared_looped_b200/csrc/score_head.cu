// Scoring head: log probabilities of given tokens under the logits
// z[v] = y . E[v] (fp32 activations y, fp16 embedding rows E[v]), the entropy of
// each row's distribution and its k most probable tokens.  The logits are never
// stored:
//   lse = log sum_v exp(z[v]),   logp(t) = z[t] - lse,
//   entropy = lse - sum_v exp(z[v] - lse) z[v]
//
// Pass 1 streams the embedding and keeps, per row and vocabulary slice, the
// running maximum m, sum l = sum e^(z - m), s = sum e^(z - m) (z - m) and the best
// candidates.  Pass 2, one CTA per row, merges the slices and decides the order
// of the best k + kSpare candidates, and the given token's logit, by fp64 dot
// products of the inputs, so the ranking does not depend on the first pass's
// rounding (ties go to the lowest token id).
#include <math_constants.h>

#include "tl_launch.cuh"

namespace tl {
namespace {

constexpr int SC_THREADS = 256;
constexpr int kSpare = 4;          // candidates kept beyond k
constexpr int kMaxCand = 16 + kSpare;

__device__ __forceinline__ bool sc_better(float x, int v, float bx, int bv) {
  return x > bx || (x == bx && v < bv);
}

// slice record of one row: m, l, s, then kc candidates (logit, id), best first
__host__ __device__ inline int rec_words(int kc) { return 3 + 2 * kc; }

// 8 rows per CTA column, a vocabulary slice per CTA row
__global__ void __launch_bounds__(SC_THREADS) score_slices_kernel(ScoreArgs a, int kc, int slices, float* rec) {
  pdl_enter();
  __shared__ float cx[SC_THREADS / 32][8][kMaxCand];
  __shared__ int cv[SC_THREADS / 32][8][kMaxCand];
  __shared__ float st[SC_THREADS / 32][8][3];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r0 = blockIdx.y * 8, rows = min(8, a.n - r0);
  const float* y0 = a.y + (size_t)r0 * a.y_stride;
  float m = -INFINITY, l = 0.f, s = 0.f;   // lane r < 8: row r
  int cnt = 0;
  const int nwarp = SC_THREADS / 32;
  const int v0 = (int)((long)a.V * blockIdx.x / slices), v1 = (int)((long)a.V * (blockIdx.x + 1) / slices);
  for (int v = v0 + warp; v < v1; v += nwarp) {
    const __half* e = a.E + (size_t)v * a.d;
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int j = 2 * lane; j < a.d; j += 64) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(e + j));
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < rows) acc[r] = fmaf(f.y, y0[r * a.y_stride + j + 1], fmaf(f.x, y0[r * a.y_stride + j], acc[r]));
    }
    float x = 0.f;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      float t = acc[r];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
      if (lane == r) x = t;
    }
    if (lane < rows) {
      if (x > m) {
        const float f = m == -INFINITY ? 0.f : expf(m - x);
        s = m == -INFINITY ? 0.f : (s + l * (m - x)) * f;
        l *= f;
        m = x;
      }
      const float e1 = expf(x - m);
      l += e1;
      s += e1 * (x - m);
      if (kc > 0 && (cnt < kc || x > cx[warp][lane][kc - 1])) {
        int p = cnt < kc ? cnt++ : kc - 1;
        while (p > 0 && x > cx[warp][lane][p - 1]) {
          cx[warp][lane][p] = cx[warp][lane][p - 1];
          cv[warp][lane][p] = cv[warp][lane][p - 1];
          --p;
        }
        cx[warp][lane][p] = x;
        cv[warp][lane][p] = v;
      }
    }
  }
  if (lane < rows) {
    for (int p = cnt; p < kc; ++p) {
      cx[warp][lane][p] = -INFINITY;
      cv[warp][lane][p] = 0x7fffffff;
    }
    st[warp][lane][0] = m;
    st[warp][lane][1] = l;
    st[warp][lane][2] = s;
  }
  __syncthreads();
  if (threadIdx.x < rows) {
    const int r = threadIdx.x;
    float M = -INFINITY, L = 0.f, S = 0.f;
    for (int w = 0; w < nwarp; ++w) M = fmaxf(M, st[w][r][0]);
    for (int w = 0; w < nwarp; ++w) {
      if (st[w][r][1] == 0.f) continue;   // no logit (a NaN sum stays)
      const float dm = st[w][r][0] - M, f = expf(dm);
      L += st[w][r][1] * f;
      S += (st[w][r][2] + st[w][r][1] * dm) * f;
    }
    float* o = rec + ((size_t)(r0 + r) * slices + blockIdx.x) * rec_words(kc);
    o[0] = M;
    o[1] = L;
    o[2] = S;
    int head[SC_THREADS / 32];
    for (int w = 0; w < nwarp; ++w) head[w] = 0;
    for (int p = 0; p < kc; ++p) {
      int bw = -1;
      float bx = -INFINITY;
      int bv = 0x7fffffff;
      for (int w = 0; w < nwarp; ++w)
        if (head[w] < kc && (bw < 0 || sc_better(cx[w][r][head[w]], cv[w][r][head[w]], bx, bv))) {
          bw = w;
          bx = cx[w][r][head[w]];
          bv = cv[w][r][head[w]];
        }
      if (bw >= 0) ++head[bw];
      o[3 + 2 * p] = bx;
      o[4 + 2 * p] = __int_as_float(bv);
    }
  }
}

constexpr int SM_THREADS = 256;

// One CTA per row: the slices' statistics and candidates merged, the chosen
// candidates and the given token scored in fp64.
__global__ void __launch_bounds__(SM_THREADS) score_merge_kernel(ScoreArgs a, int kc, int slices,
                                                                 const float* __restrict__ rec) {
  pdl_enter();
  __shared__ float wx[SM_THREADS / 32];
  __shared__ int wv[SM_THREADS / 32], wi[SM_THREADS / 32];
  __shared__ double zs[kMaxCand + 1];
  __shared__ int ids[kMaxCand + 1];
  __shared__ float red[2][SM_THREADS / 32];
  const int row = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rw = rec_words(kc);
  const float* base = rec + (size_t)row * slices * rw;
  // statistics, in a fixed order: thread-strided slices, lanes, warps
  float M = -INFINITY;
  bool nan = false;
  for (int i = tid; i < slices; i += SM_THREADS) {
    const float m = base[(size_t)i * rw];
    nan |= isnan(base[(size_t)i * rw + 1]);
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
    const float dm = m - M, f = expf(dm);
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
  const bool bad = nan || !isfinite(M) || !isfinite(L);
  const double lse = (double)M + log((double)L);
  if (tid == 0 && a.entropy) a.entropy[row] = bad ? CUDART_NAN_F : (float)(log((double)L) - (double)S / (double)L);

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

int score_slices(int n, int V) {
  const int cols = (n + 7) / 8;
  int s = cols >= 148 * 2 ? 1 : (148 * 4 + cols - 1) / cols;
  s = s > 512 ? 512 : s;
  return s > V ? V : s;
}

int score_cand(int k) { return k == 0 ? 0 : k + kSpare; }

}  // namespace

size_t score_workspace(int n, int V, int d, int k) {
  if (n == 0) return 0;
  return (size_t)n * score_slices(n, V) * rec_words(score_cand(k)) * 4 + 256;
}

tl_status launch_score_head(const ScoreArgs& a, cudaStream_t s) {
  const int kc = score_cand(a.k), slices = score_slices(a.n, a.V);
  TL_LAUNCH_PDL(score_slices_kernel, dim3(slices, (a.n + 7) / 8), SC_THREADS, 0, s, a, kc, slices, (float*)a.ws);
  TL_LAUNCH_PDL(score_merge_kernel, a.n, SM_THREADS, 0, s, a, kc, slices, (const float*)a.ws);
  return ok();
}

}  // namespace tl
