// Attention of one or a few queries a lane over a 4-bit KV cache (format:
// kv_int4.cuh):  out = softmax(q k^T / sqrt(hd)) v  with
// k, v = zero + code * scale.
//
// The queries of one key/value head (n_q tokens x the query heads that share
// it) are the eight columns of the MMA's N side, keys or head_dim elements fill
// the 16 rows:
//   S^T = K q^T : A = 16 keys x 16 head_dim elements,  B = q
//   O^T = V^T P^T : A = 16 head_dim elements x 16 keys, B = p
// Codes become fp16 values in registers (three half2 operations a pair: the
// nibble under the exponent of 1024, less the bias, times the scale plus the
// zero point; the one rounding of the value to fp16 is the read-back's own), so
// the cache is read once, as it is stored, straight from global memory: in
// the K tile lane (g, t) takes a whole 32-code group of keys g and g + 8, in
// the V tile the same 16 head_dim elements of four keys; every load instruction
// of a warp covers whole contiguous rows, and the k order inside an MMA
// is free as long as both operands agree.  A warp's next tile is requested
// before the current one is used.
//
// Bound by memory (head_dim 128: 160 bytes per key and head); about 280
// instructions per 16 keys keep the issue slots about two thirds busy at that
// rate.
//
// Work split: the context is cut into tiles of 16 keys; tile i belongs to warp
// slot i mod (CTAs of the cluster x warps), whatever the lane's length, so the
// work is even for every length and a query's arithmetic does not depend on
// the other queries of its launch: a query alone and the same query among
// several give the same bits.  Each warp keeps a running maximum and sum per
// query (base 2); the maximum is raised only when a score exceeds it by more
// than 2^8, which spares the cross-lane maximum on most tiles (weights stay
// below 2^8, well inside fp16).  The warps merge in warp order through shared
// memory, the CTAs of the cluster in rank order through distributed shared
// memory, every CTA finishing its share of the outputs: one launch, no
// workspace, the same bits at every run.
//
// Masked places never reach a sum: scores are selected, not multiplied, and
// where a key's value is not finite and some query of the tile does not see
// it, the tile's V product runs query by query with the unseen keys zeroed.
#include <algorithm>
#include <map>
#include <mutex>
#include <tuple>

#include "kv_int4.cuh"
#include "tl_launch.cuh"

namespace tl {
namespace {

constexpr int A4_COLS = 8;          // queries per CTA (MMA N)
constexpr int A4_TILE = 16;         // keys per warp tile (MMA M)
constexpr int A4_MAX_CLUSTER = 16;
constexpr float A4_SLACK = 8.f;     // the running maximum may lag by 2^8
constexpr float A4_NONE = -1e30f;   // below every score: no key yet

__device__ __forceinline__ void a4_mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 8x8 transpose of fp16 pairs across the warp
__device__ __forceinline__ uint32_t a4_transpose(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t a4_pack(float lo, float hi) {
  return kv_h2_bits(__floats2half2_rn(lo, hi));
}

__device__ __forceinline__ void a4_cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" :::
                   "memory");
}
__device__ __forceinline__ float a4_remote(const float* local, uint32_t rank) {
  uint32_t addr = (uint32_t)__cvta_generic_to_shared(local), remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote) : "memory");
  return v;
}

// Words of a row's codes that one lane holds: K, a run of head_dim / 4 codes;
// V, head_dim / 8 codes of each of four keys.
template <int HD>
struct A4 {
  static constexpr int KW = HD / 32, VW = HD / 64;
  static constexpr int KSTEPS = HD / 16, MT = HD / 16;
  static constexpr int RW = HD / 8;               // code words per row
  static constexpr int RP = HD / kInt4Group;      // parameter pairs per row
};

template <int N>
__device__ __forceinline__ void a4_load(uint32_t* r, const uint32_t* p) {
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    r[0] = v.x;
    r[1] = v.y;
    r[2] = v.z;
    r[3] = v.w;
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    r[0] = v.x;
    r[1] = v.y;
  } else {
    r[0] = *p;
  }
}

template <int HD>
struct A4Tile {
  uint32_t k[2][A4<HD>::KW], kp[2];
  uint32_t v[4][A4<HD>::VW], vp[4];
};

// a parameter pair whose values might not be finite in fp16
__device__ __forceinline__ bool a4_odd(uint32_t p) {
  return (p & 0x7fffu) >= 0x6800u || ((p >> 16) & 0x7fffu) >= 0x7800u;
}

template <int HD>
__global__ void __launch_bounds__(512) attn_int4_kernel(AttnInt4Args a) {
  using C = A4<HD>;
  pdl_enter();
  extern __shared__ __align__(16) float a4_smem[];
  const int nw = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int cls = gridDim.x, rank = blockIdx.x;
  const int ctiles = a.col_tiles, head = blockIdx.y / ctiles, c0 = (blockIdx.y % ctiles) * A4_COLS;
  const int row = blockIdx.z;
  const int cols = min(A4_COLS, a.n_q * a.group - c0);

  // the lane's cache and length
  const uint32_t *kc, *vc, *kp, *vp;
  int len;
  if (a.hdr != nullptr) {
    const int ln = a.row_lane[row];
    const char* base = a.kv_base + (size_t)(a.row_cum[row] + a.layer) * a.layer_bytes;
    kc = reinterpret_cast<const uint32_t*>(base);
    vc = reinterpret_cast<const uint32_t*>(base + a.region_bytes);
    kp = reinterpret_cast<const uint32_t*>(base + 2 * a.region_bytes);
    vp = reinterpret_cast<const uint32_t*>(base + a.region_bytes + a.layer_bytes / 2);
    len = a.hdr->pos[ln] + a.n_q;
  } else {
    kc = a.k_codes + (size_t)row * a.code_stride;
    vc = a.v_codes + (size_t)row * a.code_stride;
    kp = a.k_params + (size_t)row * a.param_stride;
    vp = a.v_params + (size_t)row * a.param_stride;
    len = a.lens[row];
  }
  len = min(len, a.max_ctx);
  kc += (size_t)head * a.max_ctx * C::RW;
  vc += (size_t)head * a.max_ctx * C::RW;
  kp += (size_t)head * a.max_ctx * C::RP;
  vp += (size_t)head * a.max_ctx * C::RP;

  // keys [first, last] seen by column c (query c / group of the lane's n_q)
  auto last_of = [&](int c) { return len - a.n_q + min(c, a.n_q * a.group - 1) / a.group; };
  auto first_of = [&](int last) { return a.window > 0 ? max(0, last - a.window + 1) : 0; };
  const int lo_all = first_of(last_of(c0)), hi_all = last_of(c0 + cols - 1);
  const int full_lo = first_of(hi_all), full_hi = last_of(c0);   // seen by every column
  int chi[2], clo[2];                                            // this lane's columns 2t, 2t + 1
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    chi[e] = last_of(c0 + min(2 * t + e, cols - 1));
    clo[e] = first_of(chi[e]);
  }

  // q as the B operand: column g, k step s = 2 jj + h covers the pairs (i, i + 4)
  // of word KW * t + jj with i = 2h (k indices 2t, 2t + 1) and 2h + 1 (+ 8)
  uint32_t qb[C::KSTEPS][2];
  {
    const int c = c0 + g, qi = c / a.group, hq = head * a.group + c % a.group;
    const bool ok = g < cols;
    const __half* q = a.q + (size_t)(row * a.n_q + (ok ? qi : 0)) * a.q_stride + (size_t)(ok ? hq : 0) * HD;
#pragma unroll
    for (int jj = 0; jj < C::KW; ++jj) {
      const uint4 w = ok ? *reinterpret_cast<const uint4*>(q + 8 * (C::KW * t + jj)) : make_uint4(0u, 0u, 0u, 0u);
      qb[2 * jj][0] = __byte_perm(w.x, w.z, 0x5410);       // elements 0, 4
      qb[2 * jj][1] = __byte_perm(w.x, w.z, 0x7632);       // 1, 5
      qb[2 * jj + 1][0] = __byte_perm(w.y, w.w, 0x5410);   // 2, 6
      qb[2 * jj + 1][1] = __byte_perm(w.y, w.w, 0x7632);   // 3, 7
    }
  }
  const float csc = rsqrtf((float)HD) * 1.4426950408889634f;   // 1/sqrt(hd) in base 2
  float m[2] = {A4_NONE, A4_NONE}, l[2] = {0.f, 0.f};
  float o[C::MT][4];
#pragma unroll
  for (int i = 0; i < C::MT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

  // MMA row r stands for key kr(r) of the tile: the four keys of a lane's V
  // pairs are then t, t + 4, t + 8, t + 12, and each load covers contiguous rows
  const int kr = (g >> 1) + 4 * (g & 1);
  const int slots = cls * nw;
  const int slot = rank * nw + warp;
  const int tile_lo = lo_all / A4_TILE;
  const int tile_hi = hi_all < 0 ? -1 : hi_all / A4_TILE;      // last tile with a key
  int tile = tile_lo + (slot - tile_lo % slots + slots) % slots;
  auto fetch = [&](int ti, A4Tile<HD>& d) {
    const int base = ti * A4_TILE;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int key = min(base + kr + 8 * h, hi_all);          // a masked place repeats the last key
      a4_load<C::KW>(d.k[h], kc + (size_t)key * C::RW + C::KW * t);
      d.kp[h] = kp[(size_t)key * C::RP + (HD == 128 ? t : t >> 1)];
    }
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const int key = min(base + t + 4 * h, hi_all);
      a4_load<C::VW>(d.v[h], vc + (size_t)key * C::RW + C::VW * g);
      d.vp[h] = vp[(size_t)key * C::RP + (HD == 128 ? g >> 1 : g >> 2)];
    }
  };

  // O^T += V^T P^T for one tile; only: -1, or the one column that takes it
  auto pv = [&](const A4Tile<HD>& d, const uint32_t* prm, uint32_t pb0, uint32_t pb1, int only) {
    const __half2 s0 = kv_bits_h2(__byte_perm(prm[0], prm[1], 0x5410)), z0 = kv_bits_h2(__byte_perm(prm[0], prm[1], 0x7632));
    const __half2 s1 = kv_bits_h2(__byte_perm(prm[2], prm[3], 0x5410)), z1 = kv_bits_h2(__byte_perm(prm[2], prm[3], 0x7632));
#pragma unroll
    for (int j = 0; j < C::VW; ++j) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        // nibbles 4hf .. 4hf + 3 of the word, keys (t, t + 4) and (t + 8, t + 12) paired
        uint32_t x0 = __byte_perm(d.v[0][j], d.v[1][j], hf ? 0x7632 : 0x5410);
        uint32_t x1 = __byte_perm(d.v[2][j], d.v[3][j], hf ? 0x7632 : 0x5410);
#pragma unroll
        for (int sel = 0; sel < 2; ++sel) {
          uint32_t af[4];
          af[0] = kv_h2_bits(__hfma2(kv_int4_pair<true>(x0), s0, z0));
          af[1] = kv_h2_bits(__hfma2(kv_int4_pair<false>(x0), s0, z0));
          af[2] = kv_h2_bits(__hfma2(kv_int4_pair<true>(x1), s1, z1));
          af[3] = kv_h2_bits(__hfma2(kv_int4_pair<false>(x1), s1, z1));
          float* acc = o[4 * j + 2 * hf + sel];
          if (only < 0) {
            a4_mma(acc, af, pb0, pb1);
          } else {
            float r[4] = {acc[0], acc[1], acc[2], acc[3]};
            a4_mma(r, af, pb0, pb1);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (2 * t + (e & 1) == only) acc[e] = r[e];
          }
          x0 >>= 8;
          x1 >>= 8;
        }
      }
    }
  };

  A4Tile<HD> cur;
  if (tile <= tile_hi) fetch(tile, cur);
  while (tile <= tile_hi) {
    const int next = tile + slots;
    A4Tile<HD> nxt;
    if (next <= tile_hi) fetch(next, nxt);
    else nxt = cur;
    // S^T = K q^T: lane (g, t) gets keys kr and kr + 8, columns 2t and 2t + 1
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    {
      const __half2 p0 = kv_bits_h2(cur.kp[0]), p1 = kv_bits_h2(cur.kp[1]);
      const __half2 s0 = __low2half2(p0), z0 = __high2half2(p0), s1 = __low2half2(p1), z1 = __high2half2(p1);
#pragma unroll
      for (int jj = 0; jj < C::KW; ++jj) {
        uint32_t x0 = cur.k[0][jj], x1 = cur.k[1][jj];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t af[4];
          af[0] = kv_h2_bits(__hfma2(kv_int4_pair<true>(x0), s0, z0));
          af[1] = kv_h2_bits(__hfma2(kv_int4_pair<true>(x1), s1, z1));
          af[2] = kv_h2_bits(__hfma2(kv_int4_pair<false>(x0), s0, z0));
          af[3] = kv_h2_bits(__hfma2(kv_int4_pair<false>(x1), s1, z1));
          a4_mma(s, af, qb[2 * jj + h][0], qb[2 * jj + h][1]);
          x0 >>= 8;
          x1 >>= 8;
        }
      }
    }
    const int base = tile * A4_TILE;
    const bool edge = base < full_lo || base + A4_TILE - 1 > full_hi;   // uniform over the CTA's lanes
    float x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = s[e] * csc;
    if (edge) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int key = base + kr + 8 * (e >> 1);
        if (key > chi[e & 1] || key < clo[e & 1]) x[e] = -INFINITY;
      }
    }
    const float mx0 = fmaxf(x[0], x[2]), mx1 = fmaxf(x[1], x[3]);
    if (__any_sync(0xffffffffu, mx0 > m[0] + A4_SLACK || mx1 > m[1] + A4_SLACK)) {
      // raise the maxima that are due, each column by its own scores alone
      float mx[2] = {mx0, mx1}, al[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], w));
        const bool up = mx[e] > m[e] + A4_SLACK;
        al[e] = up ? exp2f(m[e] - mx[e]) : 1.f;
        if (up) m[e] = mx[e];
        l[e] *= al[e];
      }
#pragma unroll
      for (int i = 0; i < C::MT; ++i) {
        o[i][0] *= al[0];
        o[i][1] *= al[1];
        o[i][2] *= al[0];
        o[i][3] *= al[1];
      }
    }
    const float p0 = exp2f(x[0] - m[0]), p1 = exp2f(x[1] - m[1]);
    const float p2 = exp2f(x[2] - m[0]), p3 = exp2f(x[3] - m[1]);
    l[0] += p0 + p2;
    l[1] += p1 + p3;
    // weights as fp16 (a rounding of 2^-11 each, of values the sum has in fp32),
    // key pairs of column g
    const uint32_t pb0 = a4_transpose(a4_pack(p0, p1)), pb1 = a4_transpose(a4_pack(p2, p3));
    bool odd = false;
    if (edge) {
#pragma unroll
      for (int h = 0; h < 4; ++h) odd |= a4_odd(cur.vp[h]);
      odd = __any_sync(0xffffffffu, odd);
    }
    if (!odd) {
      pv(cur, cur.vp, pb0, pb1, -1);
    } else {
      // some value may not be finite and some query may not see it: column by
      // column, the keys it does not see zeroed, the same arithmetic otherwise
#pragma unroll 1
      for (int c = 0; c < cols; ++c) {
        uint32_t prm[4];
        const int hi = last_of(c0 + c), lo = first_of(hi);
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const int key = base + t + 4 * h;
          prm[h] = key <= hi && key >= lo ? cur.vp[h] : 0u;
        }
        pv(cur, prm, pb0, pb1, c);
      }
    }
    cur = nxt;
    tile = next;
  }

  // ---- merge: warps (in warp order), then the cluster's CTAs (in rank order)
#pragma unroll
  for (int e = 0; e < 2; ++e)
#pragma unroll
    for (int w = 4; w < 32; w <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], w);
  // per warp [cols][HD], then per warp [cols] maxima and sums
  float* wo = a4_smem;
  float* wm = wo + (size_t)nw * cols * HD;
  float* wl = wm + nw * A4_COLS;
  float* go = wl + nw * A4_COLS;          // the CTA's record: [cols][HD], maxima, sums
  float* gm = go + cols * HD;
  float* gl = gm + A4_COLS;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int c = 2 * t + e;
    if (c < cols) {
      float* dst = wo + (size_t)(warp * cols + c) * HD + (HD / 8) * g;
#pragma unroll
      for (int i = 0; i < C::MT; ++i) *reinterpret_cast<float2*>(dst + 2 * i) = make_float2(o[i][e], o[i][e + 2]);
      if (g == 0) {
        wm[warp * A4_COLS + c] = m[e];
        wl[warp * A4_COLS + c] = l[e];
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < cols * HD; i += blockDim.x) {
    const int c = i / HD;
    float M = A4_NONE;
    for (int w = 0; w < nw; ++w) M = fmaxf(M, wm[w * A4_COLS + c]);
    float acc = 0.f, L = 0.f;
    for (int w = 0; w < nw; ++w) {
      const float f = exp2f(wm[w * A4_COLS + c] - M);
      acc = fmaf(wo[(size_t)w * cols * HD + i], f, acc);
      L = fmaf(wl[w * A4_COLS + c], f, L);
    }
    if (cls == 1) {
      const int cc = c0 + c, qi = cc / a.group, hq = head * a.group + cc % a.group;
      a.out[(size_t)(row * a.n_q + qi) * a.out_stride + (size_t)hq * HD + i % HD] =
          __float2half_rn(L == 0.f ? 0.f : acc / L);
    } else {
      go[i] = acc;
      if (i % HD == 0) {
        gm[c] = M;
        gl[c] = L;
      }
    }
  }
  if (cls == 1) return;
  a4_cluster_sync();
  // rank r finishes elements r * share .. of the record
  const int share = (cols * HD + cls - 1) / cls;
  for (int j = threadIdx.x; j < share; j += blockDim.x) {
    const int i = rank * share + j;
    if (i >= cols * HD) break;
    const int c = i / HD;
    float mr[A4_MAX_CLUSTER], lr[A4_MAX_CLUSTER], ar[A4_MAX_CLUSTER];
    float M = A4_NONE;
#pragma unroll
    for (int r = 0; r < A4_MAX_CLUSTER; ++r) {
      if (r < cls) {
        mr[r] = a4_remote(gm + c, r);
        lr[r] = a4_remote(gl + c, r);
        ar[r] = a4_remote(go + i, r);
      }
    }
#pragma unroll
    for (int r = 0; r < A4_MAX_CLUSTER; ++r)
      if (r < cls) M = fmaxf(M, mr[r]);
    float acc = 0.f, L = 0.f;
#pragma unroll
    for (int r = 0; r < A4_MAX_CLUSTER; ++r) {
      if (r < cls) {
        const float f = exp2f(mr[r] - M);
        acc = fmaf(ar[r], f, acc);
        L = fmaf(lr[r], f, L);
      }
    }
    const int cc = c0 + c, qi = cc / a.group, hq = head * a.group + cc % a.group;
    a.out[(size_t)(row * a.n_q + qi) * a.out_stride + (size_t)hq * HD + i % HD] =
        __float2half_rn(L == 0.f ? 0.f : acc / L);
  }
  a4_cluster_sync();   // no CTA leaves while another reads its shared memory
}

template <int HD>
size_t a4_smem_bytes(int nw) {
  return ((size_t)(nw + 1) * A4_COLS * HD + 2 * (size_t)(nw + 1) * A4_COLS) * sizeof(float);
}

template <int HD>
tl_status launch_a4(const AttnInt4Args& a0, cudaStream_t s) {
  static std::atomic<uint64_t> attr_done{0};
  TL_TRY(once_per_device(attr_done, []() -> tl_status {
    TL_CUDA(cudaFuncSetAttribute(attn_int4_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)a4_smem_bytes<HD>(16)));
    TL_CUDA(cudaFuncSetAttribute(attn_int4_kernel<HD>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
    return ok();
  }));
  AttnInt4Args a = a0;
  a.col_tiles = (a.n_q * a.group + A4_COLS - 1) / A4_COLS;
  int cls, nw;
  attn_int4_split(a.max_ctx, a.split_pairs * a.col_tiles, &cls, &nw);
  const dim3 grid(cls, a.H * a.col_tiles, a.n_rows);
  const cudaError_t e = launch_pdl_cluster(attn_int4_kernel<HD>, grid, dim3(32 * nw), a4_smem_bytes<HD>(nw), s,
                                           (unsigned)cls, a);
  if (e != cudaSuccess)
    return set_error(TL_ERR_CUDA, "launch of attn_int4_kernel failed: %s", cudaGetErrorString(e));
  return ok();
}

}  // namespace

// CTAs of the cluster and warps of a CTA for `pairs` (lane, head) pairs over a
// cache of max_ctx positions.
void attn_int4_split(int max_ctx, int pairs, int* cls, int* nw) {
  const int tiles = (max_ctx + A4_TILE - 1) / A4_TILE;
  *nw = tiles >= 2048 && pairs < 64 ? 16 : tiles >= 512 && pairs < 128 ? 8 : 4;
  int c = 1;
  while (c < A4_MAX_CLUSTER && c * *nw * 2 <= tiles && pairs * c * *nw < 148 * 16) c *= 2;
  *cls = c;
}

tl_status launch_attn_int4(const AttnInt4Args& a, cudaStream_t s) {
  if (a.n_rows == 0) return ok();
  if (a.hd == 128) return launch_a4<128>(a, s);
  if (a.hd == 64) return launch_a4<64>(a, s);
  return set_error(TL_ERR_UNSUPPORTED, "head_dim %d not supported", a.hd);
}

}  // namespace tl
