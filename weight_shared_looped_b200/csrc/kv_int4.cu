// Writing rows into a 4-bit KV cache and reading them back (format:
// kv_int4.cuh).
//
// Both directions move a batch of packed rows (tokens) between fp16 rows
// [n_rows][row_stride] (head h in columns [h * hd, (h + 1) * hd)) and the
// lanes' caches [H][max_ctx][hd]: row r of lane b, the (r - cu[b])-th of its
// rows, is position pos[b] + r - cu[b].  A thread owns 8 values of a row: one
// 16-byte vector of the fp16 row and one code word of the cache; the four threads
// of a group share its extremes by two shuffles.  A CTA takes consecutive rows of
// one head, so its code and parameter accesses are contiguous and its fp16
// accesses are whole head rows.
//
// Memory sets the floor: written, 4 * H * hd bytes in and 1.25 * H * hd out per
// token; read back, the reverse.  16384 tokens of 16 heads of 128 (176 MB each way)
// are written in 42 us, 4.2 TB/s (bound by issue slots: about 140 instructions per
// eight values, for the group's extremes and parameters and the rounding of each
// code), and read back in 31 us, 5.7 TB/s.  One token per lane is a launch: 2 us
// in a row of them, 6.4 us for a write and a read-back of buffers that left the caches.
#include "kv_int4.cuh"
#include "tl_launch.cuh"

namespace tl {
namespace {

constexpr int KV4_THREADS = 256;

// The lane of packed row r: the last b with cu[b] <= r (cu ascending, cu[0] =
// 0), or with cu == null the lanes' equal shares.  Returns the row's position,
// or -1 for a row behind the last lane's or outside the cache.
__device__ __forceinline__ int kv4_place(const Kv4RowsArgs& a, int r, int* lane) {
  int b, first;
  if (a.cu == nullptr) {
    const int per = a.n_rows / a.n_lanes;
    b = r / per;
    first = b * per;
  } else {
    int lo = 0, hi = a.n_lanes;   // cu[lo] <= r < cu[hi]
    if (r < __ldg(a.cu) || r >= __ldg(a.cu + a.n_lanes)) return -1;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(a.cu + mid) <= r) lo = mid;
      else hi = mid;
    }
    b = lo;
    first = __ldg(a.cu + b);
  }
  const long p = (long)__ldg(a.pos + b) + (r - first);
  *lane = b;
  return p >= 0 && p < a.max_ctx && r >= first ? (int)p : -1;
}

// U rows of K and of V per thread: their loads go out together, after one
// look-up of the CTA's rows (a look-up per thread had cost three dependent loads
// before each 16 bytes).
template <int HD, bool WRITE, int U>
__global__ void __launch_bounds__(KV4_THREADS) kv4_rows_kernel(Kv4RowsArgs a) {
  pdl_enter();
  constexpr int PARTS = HD / 8;                      // threads per row
  constexpr int ROWS = KV4_THREADS / PARTS;          // rows per pass of the CTA
  constexpr int RP = HD / kInt4Group;
  __shared__ int2 place[ROWS * U];
  const int part = threadIdx.x % PARTS, head = blockIdx.y;
  const int r0 = blockIdx.x * ROWS * U;
  for (int i = threadIdx.x; i < ROWS * U; i += KV4_THREADS) {
    int lane = 0;
    const int p = r0 + i < a.n_rows ? kv4_place(a, r0 + i, &lane) : -1;
    place[i] = make_int2(lane, p);
  }
  __syncthreads();
  const int first = threadIdx.x / PARTS;
  if (WRITE) {
    uint4 w[2][U];
    int2 at[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      at[u] = place[first + u * ROWS];
      const size_t elem = (size_t)(r0 + first + u * ROWS) * a.row_stride + (size_t)head * HD + part * 8;
#pragma unroll
      for (int z = 0; z < 2; ++z)
        w[z][u] = at[u].y >= 0 ? *reinterpret_cast<const uint4*>((z ? a.v_in : a.k_in) + elem)
                               : make_uint4(0u, 0u, 0u, 0u);
    }
    // Group extremes, least in the low half and largest (negated) in the high: one
    // reduction over the four neighbours that share a group.
    __half2 ext[2 * U];
#pragma unroll
    for (int i = 0; i < 2 * U; ++i) {
      const uint4 q = w[i % 2][i / 2];
      // NaN stays NaN
      const __half2 mn = __hmin2_nan(__hmin2_nan(kv_bits_h2(q.x), kv_bits_h2(q.y)), __hmin2_nan(kv_bits_h2(q.z), kv_bits_h2(q.w)));
      const __half2 mx = __hmax2_nan(__hmax2_nan(kv_bits_h2(q.x), kv_bits_h2(q.y)), __hmax2_nan(kv_bits_h2(q.z), kv_bits_h2(q.w)));
      ext[i] = __halves2half2(__hmin_nan(__low2half(mn), __high2half(mn)), __hneg(__hmax_nan(__low2half(mx), __high2half(mx))));
#pragma unroll
      for (int o = 1; o < 4; o <<= 1)
        ext[i] = __hmin2_nan(ext[i], kv_bits_h2(__shfl_xor_sync(0xffffffffu, kv_h2_bits(ext[i]), o)));
    }
    // Scale, zero point and reciprocal take as many instructions as a third of a
    // row's codes: the four neighbours share them out, group i to neighbour i mod 4.
    constexpr int OWN = (2 * U + 3) / 4;
    uint32_t own_param[OWN];
    float own_inv[OWN];
    const int me = threadIdx.x & 3;
#pragma unroll
    for (int j = 0; j < OWN; ++j) {
      __half2 e = ext[4 * j];
#pragma unroll
      for (int i = 1; i < 4; ++i)
        if (4 * j + i < 2 * U && me == i) e = ext[4 * j + i];
      const Int4Group g = kv_int4_group(__low2float(e), -__high2float(e));
      own_param[j] = g.param;
      own_inv[j] = g.inv;
    }
#pragma unroll
    for (int i = 0; i < 2 * U; ++i) {
      const int u = i / 2, z = i % 2;
      Int4Group g;
      g.param = __shfl_sync(0xffffffffu, own_param[i / 4], i % 4, 4);
      g.inv = __shfl_sync(0xffffffffu, own_inv[i / 4], i % 4, 4);
      g.lo = __low2float(ext[i]);
      // the eight biased codes shifted and added; their biases add up to a constant
      const uint32_t ws[4] = {w[z][u].x, w[z][u].y, w[z][u].z, w[z][u].w};
      uint32_t word = 0, bias = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 f = __half22float2(kv_bits_h2(ws[q]));
        word += kv_int4_biased(f.x, g) << (8 * q);
        word += kv_int4_biased(f.y, g) << (8 * q + 4);
        bias += (kInt4CodeBias << (8 * q)) + (kInt4CodeBias << (8 * q + 4));
      }
      word = kv_int4_marked(g) ? 0u : word - bias;
      if (at[u].y >= 0) {
        const size_t slot = (size_t)head * a.max_ctx + at[u].y;
        ((z ? a.v_codes : a.k_codes) + (size_t)at[u].x * a.code_stride)[slot * PARTS + part] = word;
        if (part % 4 == 0)
          ((z ? a.v_params : a.k_params) + (size_t)at[u].x * a.param_stride)[slot * RP + part / 4] = g.param;
      }
    }
  } else {
    uint32_t word[2][U], pr[2][U];
    int2 at[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      at[u] = place[first + u * ROWS];
      const size_t slot = (size_t)head * a.max_ctx + (at[u].y < 0 ? 0 : at[u].y);
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        word[z][u] = ((z ? a.v_codes : a.k_codes) + (size_t)at[u].x * a.code_stride)[slot * PARTS + part];
        pr[z][u] = ((z ? a.v_params : a.k_params) + (size_t)at[u].x * a.param_stride)[slot * RP + part / 4];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (at[u].y < 0) continue;
      const size_t elem = (size_t)(r0 + first + u * ROWS) * a.row_stride + (size_t)head * HD + part * 8;
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const uint32_t w = word[z][u];
        const __half2 s = __low2half2(kv_bits_h2(pr[z][u])), zr = __high2half2(kv_bits_h2(pr[z][u]));
        // pairs (i, i + 4) of the word, each value rounded once (fp16 fma)
        const uint32_t v0 = kv_h2_bits(__hfma2(kv_int4_pair<true>(w), s, zr));
        const uint32_t v1 = kv_h2_bits(__hfma2(kv_int4_pair<false>(w), s, zr));
        const uint32_t v2 = kv_h2_bits(__hfma2(kv_int4_pair<true>(w >> 8), s, zr));
        const uint32_t v3 = kv_h2_bits(__hfma2(kv_int4_pair<false>(w >> 8), s, zr));
        uint4 o;
        o.x = __byte_perm(v0, v1, 0x5410);
        o.y = __byte_perm(v2, v3, 0x5410);
        o.z = __byte_perm(v0, v1, 0x7632);
        o.w = __byte_perm(v2, v3, 0x7632);
        *reinterpret_cast<uint4*>((z ? a.v_out : a.k_out) + elem) = o;
      }
    }
  }
}

template <int HD, bool WRITE>
tl_status launch_kv4(const Kv4RowsArgs& a, cudaStream_t s) {
  constexpr int rows = KV4_THREADS / (HD / 8);
  // Two rows a thread once eight CTAs per SM are left of them (a full SM), one below.
  // Written / read, us, one and two rows a thread, 16 heads of 128:  600 rows 4.6 / 3.3
  // and 4.5 / 3.2, 1200 rows 6.2 / 4.7 and 6.6 / 4.7, 2400 rows 9.4 / 7.0 and 9.2 / 6.3,
  // 16384 rows 46.3 / 34.6 and 42.2 / 30.9.  Four rows: 8.1 / 4.6 at 1200, 43.2 / 31.6
  // at 16384.
  if ((long)a.n_rows * a.H >= (long)rows * 2 * 148 * 8)
    TL_LAUNCH_PDL((kv4_rows_kernel<HD, WRITE, 2>), dim3((a.n_rows + 2 * rows - 1) / (2 * rows), a.H), KV4_THREADS, 0, s, a);
  else
    TL_LAUNCH_PDL((kv4_rows_kernel<HD, WRITE, 1>), dim3((a.n_rows + rows - 1) / rows, a.H), KV4_THREADS, 0, s, a);
  return ok();
}

}  // namespace

tl_status launch_kv4_rows(const Kv4RowsArgs& a, bool write, cudaStream_t s) {
  if (a.n_rows == 0) return ok();
  if (a.hd == 128) return write ? launch_kv4<128, true>(a, s) : launch_kv4<128, false>(a, s);
  if (a.hd == 64) return write ? launch_kv4<64, true>(a, s) : launch_kv4<64, false>(a, s);
  return set_error(TL_ERR_UNSUPPORTED, "head_dim %d not supported", a.hd);
}

}  // namespace tl
