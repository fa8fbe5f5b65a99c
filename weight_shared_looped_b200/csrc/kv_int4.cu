// Writing rows into a 4-bit KV cache and reading them back (format:
// kv_int4.cuh).
//
// Both directions move a batch of packed rows (tokens) between fp16 rows
// [n_rows][row_stride] (head h in columns [h * hd, (h + 1) * hd)) and the
// lanes' caches [H][max_ctx][hd]: row r of lane b, the (r - cu[b])-th of its
// rows, is position pos[b] + r - cu[b].  A thread owns 8 values: one 16-byte
// vector of the fp16 row and one code word of the cache; the four threads of a
// group share its extremes by two shuffles.  Consecutive threads take
// consecutive positions of one head, so a CTA's code and parameter accesses
// are contiguous and its fp16 accesses are whole head rows.
//
// Bound by memory: written, 4 * H * hd bytes in and 1.25 * H * hd out per
// token; read back, the reverse.
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

template <int HD, bool WRITE>
__global__ void __launch_bounds__(KV4_THREADS) kv4_rows_kernel(Kv4RowsArgs a) {
  pdl_enter();
  constexpr int PARTS = HD / 8;                      // threads per row
  constexpr int ROWS = KV4_THREADS / PARTS;          // rows per CTA
  const int part = threadIdx.x % PARTS, head = blockIdx.y;
  const bool is_v = blockIdx.z != 0;
  const int r = blockIdx.x * ROWS + threadIdx.x / PARTS;
  int lane = 0;
  const int p = r < a.n_rows ? kv4_place(a, r, &lane) : -1;
  uint32_t* codes = (is_v ? a.v_codes : a.k_codes) + (size_t)lane * a.code_stride;
  uint32_t* params = (is_v ? a.v_params : a.k_params) + (size_t)lane * a.param_stride;
  const size_t slot = (size_t)head * a.max_ctx + (p < 0 ? 0 : p);
  const size_t elem = (size_t)(r < a.n_rows ? r : 0) * a.row_stride + (size_t)head * HD + part * 8;
  if (WRITE) {
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if (p >= 0) w = *reinterpret_cast<const uint4*>((is_v ? a.v_in : a.k_in) + elem);
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
    __half2 mn = kv_bits_h2(ws[0]), mx = mn;
#pragma unroll
    for (int i = 1; i < 4; ++i) {                    // NaN stays NaN
      mn = __hmin2_nan(mn, kv_bits_h2(ws[i]));
      mx = __hmax2_nan(mx, kv_bits_h2(ws[i]));
    }
    // the four threads of a group are neighbours
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      mn = __hmin2_nan(mn, kv_bits_h2(__shfl_xor_sync(0xffffffffu, kv_h2_bits(mn), o)));
      mx = __hmax2_nan(mx, kv_bits_h2(__shfl_xor_sync(0xffffffffu, kv_h2_bits(mx), o)));
    }
    if (p < 0) return;
    const Int4Group g = kv_int4_group(__half2float(__hmin_nan(__low2half(mn), __high2half(mn))),
                                      __half2float(__hmax_nan(__low2half(mx), __high2half(mx))));
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(kv_bits_h2(ws[i]));
      word |= kv_int4_code(f.x, g) << (8 * i);
      word |= kv_int4_code(f.y, g) << (8 * i + 4);
    }
    codes[slot * PARTS + part] = word;
    if (part % 4 == 0) params[slot * (HD / kInt4Group) + part / 4] = g.param;
  } else {
    if (p < 0) return;
    const uint32_t word = codes[slot * PARTS + part];
    const __half2 pr = kv_bits_h2(params[slot * (HD / kInt4Group) + part / 4]);
    const __half2 s = __low2half2(pr), z = __high2half2(pr);
    // pairs (i, i + 4) of the word, each value rounded once (fp16 fma)
    const uint32_t v0 = kv_h2_bits(__hfma2(kv_int4_pair<true>(word), s, z));
    const uint32_t v1 = kv_h2_bits(__hfma2(kv_int4_pair<false>(word), s, z));
    const uint32_t v2 = kv_h2_bits(__hfma2(kv_int4_pair<true>(word >> 8), s, z));
    const uint32_t v3 = kv_h2_bits(__hfma2(kv_int4_pair<false>(word >> 8), s, z));
    uint4 o;
    o.x = __byte_perm(v0, v1, 0x5410);
    o.y = __byte_perm(v2, v3, 0x5410);
    o.z = __byte_perm(v0, v1, 0x7632);
    o.w = __byte_perm(v2, v3, 0x7632);
    *reinterpret_cast<uint4*>((is_v ? a.v_out : a.k_out) + elem) = o;
  }
}

}  // namespace

tl_status launch_kv4_rows(const Kv4RowsArgs& a, bool write, cudaStream_t s) {
  if (a.n_rows == 0) return ok();
  const int rows = KV4_THREADS / (a.hd / 8);
  const dim3 grid((a.n_rows + rows - 1) / rows, a.H, 2);
  if (a.hd == 128) {
    if (write) TL_LAUNCH_PDL((kv4_rows_kernel<128, true>), grid, KV4_THREADS, 0, s, a);
    else TL_LAUNCH_PDL((kv4_rows_kernel<128, false>), grid, KV4_THREADS, 0, s, a);
  } else if (a.hd == 64) {
    if (write) TL_LAUNCH_PDL((kv4_rows_kernel<64, true>), grid, KV4_THREADS, 0, s, a);
    else TL_LAUNCH_PDL((kv4_rows_kernel<64, false>), grid, KV4_THREADS, 0, s, a);
  } else {
    return set_error(TL_ERR_UNSUPPORTED, "head_dim %d not supported", a.hd);
  }
  return ok();
}

}  // namespace tl
