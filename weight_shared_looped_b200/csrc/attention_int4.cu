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
// the cache is read once, as it is stored: each warp copies its tiles of 32 keys
// (5 KB for head_dim 128) through a ring of its own in shared memory, one tile
// ahead of the one it works on (loads into registers instead left a warp waiting
// for memory at every tile: 1.3 us per 16 keys against 0.2 of work).  Sixteen
// warps per SM keep 80 KB on the way, which covers the memory's latency; rings of
// three and four tiles measured the same or slower, and tiles of 16 keys 48 us
// where 32 take 41.  From the K tile lane (g, t) takes a whole 32-code group of
// two keys, from the V tile the same 16 head_dim elements of four keys; the k
// order inside an MMA is free as long as both operands agree, and is chosen so
// that no read has a bank conflict.
//
// Memory sets the floor (head_dim 128: 160 bytes per key and head), the issue
// slots the pace: about 340 instructions per 16 keys, 63 % of the slots busy.
// Two lanes of up to 65536 positions, 8 cache heads, 4 queries per head: 147 MB in
// 41 us, 3.6 TB/s.  Many short lanes are bound by their launch, the merge and the tail.
//
// Work split: the context is cut into tiles of 32 keys; tile i belongs to slot i mod
// slots, whatever the lane's length, so the work is even for every length.  For a
// given split the other queries of a launch do not change a query's arithmetic; a
// caller's split follows from max_ctx and the number of lanes, heads and column tiles
// (eight queries x query heads each), a model's from max_ctx alone.  A warp takes a slot,
// or some in turn, and keeps a running reference and sum per query (base 2); the reference
// is raised only when a weight would pass 2^15 (A4_SLACK), which spares the cross-lane
// maximum on most tiles.  The slots' records are joined in a fixed order through shared memory, the CTAs of a cluster
// through distributed shared memory, every CTA finishing its share of the outputs: one
// launch, no workspace.  The longest contexts are split over more CTAs, whose records
// a second launch joins.  The bits are the same at every run.
//
// A model's decode step makes its new entry here (FUSED): RoPE of q in every CTA, of k
// in the one that reads the entry's tile, which quantises and appends it, while the
// other tiles are on their way: a launch less per layer (one lane of 384 positions, 10
// layer applications: 309 -> 284 us per step).
//
// Masked places never reach a sum: scores are selected, not multiplied, and
// where a key's value is not finite and some query of the tile does not see
// it, the tile's V product runs query by query with the unseen keys zeroed.
#include <algorithm>

#include "kv_int4.cuh"
#include "tl_launch.cuh"

namespace tl {
namespace {

constexpr int A4_COLS = 8;          // queries per CTA (MMA N)
constexpr int A4_TILE = 32;         // keys per warp tile: two sub-tiles of 16 (MMA M)
constexpr int A4_GROUP = 4;          // slots whose records are joined first
constexpr int A4_WIDE = 12;          // warps of a CTA that has an SM to itself; others have 4
constexpr int A4_MAX_CLUSTER = 8;
constexpr int A4_MAX_SPLIT = 64;
constexpr int A4_MAX_SMEM = 226 * 1024;   // beside the static array
constexpr int A4_STAGES = 2;         // tiles of a warp's ring
// A softmax weight is 2^(score - m) with m 7 below a score that was the largest when it was
// set, and m is raised when a score exceeds it by more than 15: the largest weight lies
// between 2^7 and 2^15, so that in fp16 weights down to 2^-21 of it keep all their bits and
// those down to 2^-32 of it count (with m at the largest score, keys below 2^-25 of it
// vanished from the products while the sum had them).
constexpr float A4_LIFT = 7.f, A4_SLACK = 15.f;
constexpr float A4_NONE = -1e30f;   // below every score: no key yet

__device__ __forceinline__ void a4_mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float a4_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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
// V, head_dim / 8 codes of each of four keys.  A tile in shared memory: K rows, V
// rows, K parameters, V parameters, as the cache has them; of the V rows, those
// with bit 2 set have their 16-byte pieces swapped in pairs.
template <int HD>
struct A4 {
  static constexpr int KW = HD / 32, VW = HD / 64;
  static constexpr int KSTEPS = HD / 16, MT = HD / 16;
  static constexpr int RW = HD / 8;               // code words per row
  static constexpr int RP = HD / kInt4Group;      // parameter pairs per row
  static constexpr int V0 = A4_TILE * RW, KP0 = 2 * V0, VP0 = KP0 + A4_TILE * RP;
  static constexpr int WORDS = VP0 + A4_TILE * RP;   // words of a tile
  static constexpr int VSWAP = HD == 128 ? 8 : 0;    // word index bit the swap flips
};

template <int N>
__device__ __forceinline__ void a4_lds(uint32_t* r, const uint32_t* p) {
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

__device__ __forceinline__ void a4_copy16(uint32_t* dst, const uint32_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}

// a parameter pair whose values might not be finite in fp16
__device__ __forceinline__ bool a4_odd(uint32_t p) {
  return (p & 0x7fffu) >= 0x6800u || ((p >> 16) & 0x7fffu) >= 0x7800u;
}

__device__ __forceinline__ void a4_copy4(uint32_t* dst, const uint32_t* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}

// A query's output from its weighted sum and the sum of its weights.  One that sees no key
// gets zeros; where all of its scores are -inf (an infinite query) there is no distribution:
// NaN.
__device__ __forceinline__ __half a4_output(float acc, float L, bool sees) {
  return __float2half_rn(L == 0.f ? (sees ? CUDART_NAN_F : 0.f) : acc / L);
}

template <int HD, int WARPS, bool FUSED>
__global__ void __launch_bounds__(32 * WARPS, WARPS == A4_WIDE ? 1 : 4) attn_int4_kernel(AttnInt4Args a) {
  using C = A4<HD>;
  // What a model's decode reads before pdl_enter() (positions, the cache) was written
  // before the QKV projection it waits for there, which has itself waited for that.
  if (!FUSED) pdl_enter();
  extern __shared__ __align__(128) float a4_smem[];
  __shared__ __align__(16) __half a4_q[FUSED ? HD : 8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
  len = max(0, min(len, a.max_ctx));
  kc += (size_t)head * a.max_ctx * C::RW;
  vc += (size_t)head * a.max_ctx * C::RW;
  kp += (size_t)head * a.max_ctx * C::RP;
  vp += (size_t)head * a.max_ctx * C::RP;

  // keys [first, last] seen by column c (query c / group of the lane's n_q)
  auto last_of = [&](int c) { return len - a.n_q + min(c, a.n_q * a.group - 1) / a.group; };
  auto first_of = [&](int last) { return a.window > 0 ? max(0, last - a.window + 1) : 0; };
  const int lo_all = first_of(last_of(c0)), hi_all = last_of(c0 + cols - 1);
  const int full_lo = first_of(hi_all), full_hi = last_of(c0);   // seen by every column

  const float csc = rsqrtf((float)HD) * 1.4426950408889634f;   // 1/sqrt(hd) in base 2
  float m[2], l[2], o[C::MT][4];

  // MMA row r stands for key kr(r) of the tile: a lane's V pairs are then the keys
  // kr(2t), kr(2t + 1) and those + 8, and the reads of a quarter (half) warp fall on
  // distinct banks
  const int kr = g ^ ((g >> 1) & 1);
  const int vk[4] = {2 * t ^ (t & 1), (2 * t + 1) ^ (t & 1), (2 * t ^ (t & 1)) + 8, ((2 * t + 1) ^ (t & 1)) + 8};
  // slot s takes tiles s, s + slots, ..; this warp takes `passes` slots in turn
  const int passes = WARPS == A4_WIDE ? a.passes : 1;
  const int stride = cls * WARPS, slots = stride * passes;
  const int tile_lo = lo_all / A4_TILE;
  const int tile_hi = hi_all < 0 ? -1 : hi_all / A4_TILE;      // last tile with a key
  auto first_tile = [&](int pass) {
    return tile_lo + (pass * stride + rank * WARPS + warp - tile_lo % slots + slots) % slots;
  };
  uint32_t* ring = reinterpret_cast<uint32_t*>(a4_smem) + (size_t)warp * A4_STAGES * C::WORDS;
  // head_dim 64 with an odd max_ctx, or a caller's strides, leave parameters on 4 bytes
  const bool par16 = (((uintptr_t)kp | (uintptr_t)vp) & 15) == 0;
  // copies tile ti into its ring slot: whole 16-byte pieces, in the order of memory;
  // where the cache ends inside the tile its last row repeats
  auto fetch = [&](int ti, int slot_) {
    uint32_t* dst = ring + slot_ * C::WORDS;
    const int base = ti * A4_TILE;
    constexpr int PR = C::RW / 4;                  // pieces per code row
    constexpr int NP = A4_TILE * C::RP / 4;        // 16-byte pieces of K's parameters (and of V's)
    if (par16 && base + A4_TILE <= a.max_ctx) {
      const uint32_t* sk = kc + (size_t)base * C::RW + 4 * lane;
      const uint32_t* sv = vc + (size_t)base * C::RW + 4 * lane;
      // the row of piece lane + 32 i has the swap bit of row lane / PR (32 pieces are 8 or 16 rows)
      uint32_t* dv = dst + C::V0 + ((4 * lane) ^ ((lane / PR) & 4 ? C::VSWAP : 0));
#pragma unroll
      for (int i = 0; i < A4_TILE * PR / 32; ++i) {
        a4_copy16(dst + 4 * lane + 128 * i, sk + 128 * i);
        a4_copy16(dv + 128 * i, sv + 128 * i);
      }
#pragma unroll
      for (int i = 0; i < (NP + 31) / 32; ++i)
        if (lane < NP) {
          a4_copy16(dst + C::KP0 + 4 * lane, kp + (size_t)base * C::RP + 4 * lane);
          a4_copy16(dst + C::VP0 + 4 * lane, vp + (size_t)base * C::RP + 4 * lane);
        }
    } else {
      const int last = a.max_ctx - 1;
#pragma unroll 1
      for (int p = lane; p < A4_TILE * PR; p += 32) {
        const int r = p / PR, c = p % PR;
        const size_t src = (size_t)min(base + r, last) * C::RW + 4 * c;
        a4_copy16(dst + 4 * p, kc + src);
        a4_copy16(dst + C::V0 + r * C::RW + ((4 * c) ^ ((r & 4) ? C::VSWAP : 0)), vc + src);
      }
#pragma unroll 1
      for (int p = lane; p < A4_TILE * C::RP; p += 32) {
        const size_t src = (size_t)min(base + p / C::RP, last) * C::RP + p % C::RP;
        a4_copy4(dst + C::KP0 + p, kp + src);
        a4_copy4(dst + C::VP0 + p, vp + src);
      }
    }
  };

  // O^T += V^T P^T for one sub-tile; only: -1, or the one column that takes it
  auto pv = [&](const uint32_t* tw, int sub, const uint32_t* prm, uint32_t pb0, uint32_t pb1, int only) {
    uint32_t dv[4][C::VW];
#pragma unroll
    for (int h = 0; h < 4; ++h)
      a4_lds<C::VW>(dv[h], tw + C::V0 + (16 * sub + vk[h]) * C::RW + ((C::VW * g) ^ ((vk[h] & 4) ? C::VSWAP : 0)));
    const __half2 s0 = kv_bits_h2(__byte_perm(prm[0], prm[1], 0x5410)), z0 = kv_bits_h2(__byte_perm(prm[0], prm[1], 0x7632));
    const __half2 s1 = kv_bits_h2(__byte_perm(prm[2], prm[3], 0x5410)), z1 = kv_bits_h2(__byte_perm(prm[2], prm[3], 0x7632));
#pragma unroll
    for (int j = 0; j < C::VW; ++j) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        // nibbles 4hf .. 4hf + 3 of the word, the lane's keys paired
        uint32_t x0 = __byte_perm(dv[0][j], dv[1][j], hf ? 0x7632 : 0x5410);
        uint32_t x1 = __byte_perm(dv[2][j], dv[3][j], hf ? 0x7632 : 0x5410);
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
          if (sel == 0) {
            x0 >>= 8;
            x1 >>= 8;
          }
        }
      }
    }
  };

  // records of the slots [passes][WARPS][cols][HD] (over the rings when there is one
  // pass), their maxima and sums, the groups', the CTA's record
  const int my_slots = passes * WARPS, my_groups = my_slots / A4_GROUP, elems = cols * HD;
  float* rec = a4_smem + (passes > 1 ? WARPS * A4_STAGES * C::WORDS : 0);
  float* rm = rec + (size_t)my_slots * elems;
  float* rl = rm + my_slots * cols;
  float* gm = rl + my_slots * cols;
  float* gl = gm + my_groups * cols;
  float* go = gl + my_groups * cols;
  float* cm = go + elems;
  float* cl = cm + cols;

  int pass = 0, tile = first_tile(0), ahead_pass = 0, ahead = tile, in_slot = 0, out_slot = 0;
  auto request = [&]() {                           // one group per tile, empty behind the last
    while (ahead > tile_hi && ahead_pass + 1 < passes) ahead = first_tile(++ahead_pass);
    if (ahead <= tile_hi) fetch(ahead, in_slot);
    asm volatile("cp.async.commit_group;" ::: "memory");
    ahead += slots;
    in_slot = in_slot + 1 == A4_STAGES ? 0 : in_slot + 1;
  };
  // the tile that takes the new entry waits for it, the others' first copies do not
  const bool holds_new = FUSED && ahead == tile_hi;
  if (!holds_new)
#pragma unroll
    for (int i = 0; i < A4_STAGES - 1; ++i) request();
  if constexpr (FUSED) {
    const int pos = hi_all;
    float2 cs[HD / 64];
#pragma unroll
    for (int p = 0; p < HD / 64; ++p) cs[p] = a.rope_cs[(size_t)pos * (HD / 2) + lane + 32 * p];
    pdl_enter();
    // rotate-half pairs (i, i + HD / 2), i = lane + 32 p, of q (every CTA, warp 0) and of
    // k, with v (warp 1 of the CTA that reads the new entry's tile)
    const float* x = a.qkv + (size_t)row * 3 * a.H * HD + (size_t)head * HD + lane;
    if (warp == 0) {
#pragma unroll
      for (int p = 0; p < HD / 64; ++p) {
        const float2 r = kv_rope(__ldcg(x + 32 * p), __ldcg(x + 32 * p + HD / 2), cs[p]);
        a4_q[lane + 32 * p] = __float2half_rn(r.x);
        a4_q[lane + 32 * p + HD / 2] = __float2half_rn(r.y);
      }
    } else if (warp == 1 && tile_hi % slots % stride / WARPS == rank) {
      const float *k = x + (size_t)a.H * HD, *v = k + (size_t)a.H * HD;
      __half kh[HD / 64][2], vh[HD / 64][2];
#pragma unroll
      for (int p = 0; p < HD / 64; ++p) {
        const float2 r = kv_rope(__ldcg(k + 32 * p), __ldcg(k + 32 * p + HD / 2), cs[p]);
        kh[p][0] = __float2half_rn(r.x);
        kh[p][1] = __float2half_rn(r.y);
        vh[p][0] = __float2half_rn(__ldcg(v + 32 * p));
        vh[p][1] = __float2half_rn(__ldcg(v + 32 * p + HD / 2));
      }
      // the cache is const to the rest of the kernel: this row is read behind the barrier only
      uint32_t *ck = const_cast<uint32_t*>(kc) + (size_t)pos * C::RW, *cv = const_cast<uint32_t*>(vc) + (size_t)pos * C::RW;
      uint32_t *pk = const_cast<uint32_t*>(kp) + (size_t)pos * C::RP, *pv_ = const_cast<uint32_t*>(vp) + (size_t)pos * C::RP;
#pragma unroll
      for (int p = 0; p < HD / 64; ++p)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const int grp = p + hh * (HD / 64);
          kv_int4_append_group(kh[p][hh], vh[p][hh], ck + 4 * grp, cv + 4 * grp, pk + grp, pv_ + grp);
        }
      __threadfence_block();
    }
    __syncthreads();
    if (holds_new)
#pragma unroll
      for (int i = 0; i < A4_STAGES - 1; ++i) request();
  }
  // q as the B operand: column g, k step s = 2 jj + h covers the pairs (i, i + 4)
  // of word KW * t + jj with i = 2h (k indices 2t, 2t + 1) and 2h + 1 (+ 8)
  uint32_t qb[C::KSTEPS][2];
  {
    const int c = c0 + g, qi = c / a.group, hq = head * a.group + c % a.group;
    const bool ok = g < cols;
    const __half* q = FUSED ? a4_q : a.q + (size_t)(row * a.n_q + (ok ? qi : 0)) * a.q_stride + (size_t)(ok ? hq : 0) * HD;
#pragma unroll
    for (int jj = 0; jj < C::KW; ++jj) {
      const uint4 w = ok ? *reinterpret_cast<const uint4*>(q + 8 * (C::KW * t + jj)) : make_uint4(0u, 0u, 0u, 0u);
      qb[2 * jj][0] = __byte_perm(w.x, w.z, 0x5410);       // elements 0, 4
      qb[2 * jj][1] = __byte_perm(w.x, w.z, 0x7632);       // 1, 5
      qb[2 * jj + 1][0] = __byte_perm(w.y, w.w, 0x5410);   // 2, 6
      qb[2 * jj + 1][1] = __byte_perm(w.y, w.w, 0x7632);   // 3, 7
    }
  }
#pragma unroll 1
  while (true) {
    m[0] = m[1] = A4_NONE;
    l[0] = l[1] = 0.f;
#pragma unroll
    for (int i = 0; i < C::MT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
#pragma unroll 1
    for (; tile <= tile_hi; tile += slots) {
      asm volatile("cp.async.wait_group %0;" ::"n"(A4_STAGES - 2) : "memory");
      __syncwarp();                                  // every lane's copies of this tile; the slot before is free
      request();
      const uint32_t* tw = ring + out_slot * C::WORDS;
      out_slot = out_slot + 1 == A4_STAGES ? 0 : out_slot + 1;
      // S^T = K q^T: lane (g, t) gets keys kr and kr + 8 of each sub-tile, columns 2t and 2t + 1
      float s[2][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        s[u][0] = s[u][1] = s[u][2] = s[u][3] = 0.f;
        const int r0 = 16 * u + kr, r1 = r0 + 8;
        uint32_t k0[C::KW], k1[C::KW];
        a4_lds<C::KW>(k0, tw + r0 * C::RW + C::KW * t);
        a4_lds<C::KW>(k1, tw + r1 * C::RW + C::KW * t);
        const __half2 p0 = kv_bits_h2(tw[C::KP0 + r0 * C::RP + (HD == 128 ? t : t >> 1)]);
        const __half2 p1 = kv_bits_h2(tw[C::KP0 + r1 * C::RP + (HD == 128 ? t : t >> 1)]);
        const __half2 s0 = __low2half2(p0), z0 = __high2half2(p0), s1 = __low2half2(p1), z1 = __high2half2(p1);
#pragma unroll
        for (int jj = 0; jj < C::KW; ++jj) {
          uint32_t x0 = k0[jj], x1 = k1[jj];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t af[4];
            af[0] = kv_h2_bits(__hfma2(kv_int4_pair<true>(x0), s0, z0));
            af[1] = kv_h2_bits(__hfma2(kv_int4_pair<true>(x1), s1, z1));
            af[2] = kv_h2_bits(__hfma2(kv_int4_pair<false>(x0), s0, z0));
            af[3] = kv_h2_bits(__hfma2(kv_int4_pair<false>(x1), s1, z1));
            a4_mma(s[u], af, qb[2 * jj + h][0], qb[2 * jj + h][1]);
            if (h == 0) {
              x0 >>= 8;
              x1 >>= 8;
            }
          }
        }
      }
      const int base = tile * A4_TILE;
      const bool edge = base < full_lo || base + A4_TILE - 1 > full_hi;   // uniform over the warp
      if (edge) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int hi = last_of(c0 + min(2 * t + (e & 1), cols - 1)), lo = first_of(hi);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int key = base + 16 * u + kr + 8 * (e >> 1);
            if (key > hi || key < lo) s[u][e] = -INFINITY;
          }
        }
      }
      const float mx0 = fmaxf(fmaxf(s[0][0], s[0][2]), fmaxf(s[1][0], s[1][2]));
      const float mx1 = fmaxf(fmaxf(s[0][1], s[0][3]), fmaxf(s[1][1], s[1][3]));
      if (__any_sync(0xffffffffu, mx0 * csc > m[0] + A4_SLACK || mx1 * csc > m[1] + A4_SLACK)) {
        // raise the maxima that are due, each column by its own scores alone
        float mx[2] = {mx0, mx1}, al[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int w = 4; w < 32; w <<= 1) mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], w));
          mx[e] *= csc;
          const bool up = mx[e] > m[e] + A4_SLACK;
          al[e] = up ? a4_ex2(m[e] - (mx[e] - A4_LIFT)) : 1.f;
          if (up) m[e] = mx[e] - A4_LIFT;
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
      // weights as fp16 (a rounding of 2^-11 each, 2^-32 of the largest where they are
      // subnormal, of values the sum has in fp32), key pairs of column g
      uint32_t pb[2][2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float p0 = a4_ex2(fmaf(s[u][0], csc, -m[0])), p1 = a4_ex2(fmaf(s[u][1], csc, -m[1]));
        const float p2 = a4_ex2(fmaf(s[u][2], csc, -m[0])), p3 = a4_ex2(fmaf(s[u][3], csc, -m[1]));
        l[0] += p0 + p2;
        l[1] += p1 + p3;
        pb[u][0] = a4_transpose(a4_pack(p0, p1));
        pb[u][1] = a4_transpose(a4_pack(p2, p3));
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t prm[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) prm[h] = tw[C::VP0 + (16 * u + vk[h]) * C::RP + (HD == 128 ? g >> 1 : g >> 2)];
        // keys that no query sees may hold anything: they count as zero
        bool odd = false;
        if (edge) {
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const int key = base + 16 * u + vk[h];
            if (key > hi_all || key < lo_all) prm[h] = 0u;
            odd |= a4_odd(prm[h]);
          }
          odd = __any_sync(0xffffffffu, odd);
        }
        if (!odd) {
          pv(tw, u, prm, pb[u][0], pb[u][1], -1);
        } else {
          // some value may not be finite and some query may not see it: column by
          // column, the keys it does not see zeroed, the same arithmetic otherwise
#pragma unroll 1
          for (int c = 0; c < cols; ++c) {
            uint32_t own[4];
            const int hi = last_of(c0 + c), lo = first_of(hi);
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              const int key = base + 16 * u + vk[h];
              own[h] = key <= hi && key >= lo ? prm[h] : 0u;
            }
            pv(tw, u, own, pb[u][0], pb[u][1], c);
          }
        }
      }
    }
    if (passes == 1) __syncthreads();              // the rings' memory holds the records from here on
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int w = 4; w < 32; w <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], w);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int c = 2 * t + e;
      if (c < cols) {
        const int r = (pass * WARPS + warp) * cols + c;
        float* dst = rec + (size_t)r * HD + (HD / 8) * g;
#pragma unroll
        for (int i = 0; i < C::MT; ++i) *reinterpret_cast<float2*>(dst + 2 * i) = make_float2(o[i][e], o[i][e + 2]);
        if (g == 0) {
          rm[r] = m[e];
          rl[r] = l[e];
        }
      }
    }
    if (++pass == passes) break;
    tile = first_tile(pass);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();

  // ---- join: the slots of a group in their order, the groups, the cluster's CTAs.
  // The join of one record has its bits, so a group per CTA and all groups in one CTA
  // give the same.
  auto group_record = [&](int r0, int i, float* M, float* acc, float* L) {
    const int c = i / HD;
    *M = A4_NONE;
    *acc = *L = 0.f;
#pragma unroll
    for (int w = 0; w < A4_GROUP; ++w) *M = fmaxf(*M, rm[(r0 + w) * cols + c]);
#pragma unroll
    for (int w = 0; w < A4_GROUP; ++w) {
      const float f = exp2f(rm[(r0 + w) * cols + c] - *M);
      *acc = fmaf(rec[(size_t)(r0 + w) * elems + i], f, *acc);
      *L = fmaf(rl[(r0 + w) * cols + c], f, *L);
    }
  };
  auto to_output = [&](int i, float acc, float L) {
    const int cc = c0 + i / HD, qi = cc / a.group, hq = head * a.group + cc % a.group;
    a.out[(size_t)(row * a.n_q + qi) * a.out_stride + (size_t)hq * HD + i % HD] = a4_output(acc, L, FUSED || last_of(cc) >= 0);
  };
  // a split beyond a cluster: record `all` of `of` goes to the merge kernel
  auto to_workspace = [&](int all, int of, int i, float M, float acc, float L) {
    const int c = i / HD;
    float* to = a.ws + (((size_t)row * gridDim.y + blockIdx.y) * of + all) * (A4_COLS * (HD + 2));
    to[i] = acc;
    if (i % HD == 0) {
      to[A4_COLS * HD + c] = M;
      to[A4_COLS * HD + A4_COLS + c] = L;
    }
  };
  auto to_cluster = [&](int i, float M, float acc, float L) {
    go[i] = acc;
    if (i % HD == 0) {
      cm[i / HD] = M;
      cl[i / HD] = L;
    }
  };
  if constexpr (WARPS == A4_GROUP) {
    for (int i = threadIdx.x; i < elems; i += blockDim.x) {
      float M, acc, L;
      group_record(0, i, &M, &acc, &L);
      if (cls == 1) to_output(i, acc, L);
      else if (a.ws != nullptr) to_workspace(rank, cls, i, M, acc, L);
      else to_cluster(i, M, acc, L);
    }
  } else {
    constexpr int WG = WARPS / A4_GROUP;           // groups of a pass
    for (int gg = warp / A4_GROUP; gg < my_groups; gg += WG) {
      for (int i = threadIdx.x % (32 * A4_GROUP); i < elems; i += 32 * A4_GROUP) {
        float M, acc, L;
        group_record(gg * A4_GROUP, i, &M, &acc, &L);
        if (a.ws != nullptr) {
          to_workspace(gg / WG * (cls * WG) + rank * WG + gg % WG, cls * my_groups, i, M, acc, L);
          continue;
        }
        rec[(size_t)gg * A4_GROUP * elems + i] = acc;   // over the group's first, which this thread alone reads
        if (i % HD == 0) {
          gm[gg * cols + i / HD] = M;
          gl[gg * cols + i / HD] = L;
        }
      }
    }
    if (a.ws != nullptr) return;
    __syncthreads();
    for (int i = threadIdx.x; i < elems; i += blockDim.x) {
      const int c = i / HD;
      float M = A4_NONE, acc = 0.f, L = 0.f;
#pragma unroll 3
      for (int gg = 0; gg < my_groups; ++gg) M = fmaxf(M, gm[gg * cols + c]);
#pragma unroll 3
      for (int gg = 0; gg < my_groups; ++gg) {
        const float f = exp2f(gm[gg * cols + c] - M);
        acc = fmaf(rec[(size_t)gg * A4_GROUP * elems + i], f, acc);
        L = fmaf(gl[gg * cols + c], f, L);
      }
      if (cls == 1) to_output(i, acc, L);
      else to_cluster(i, M, acc, L);
    }
  }
  if (cls == 1 || a.ws != nullptr) return;
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
        mr[r] = a4_remote(cm + c, r);
        lr[r] = a4_remote(cl + c, r);
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
    to_output(i, acc, L);
  }
  a4_cluster_sync();   // no CTA leaves while another reads its shared memory
}

// Joins the records of a split in their order: a CTA per query and head, two
// threads per output element, each with half of the records, all of them
// requested at once.
template <int HD>
__global__ void __launch_bounds__(2 * HD) attn_int4_merge_kernel(AttnInt4Args a, int splits) {
  pdl_enter();
  const int cols_all = a.n_q * a.group;
  const int head = blockIdx.x / cols_all, cc = blockIdx.x % cols_all, row = blockIdx.y;
  const int c = cc % A4_COLS;
  constexpr int REC = A4_COLS * (HD + 2), HALF = A4_MAX_SPLIT / 2;
  const float* rec =
      a.ws + (((size_t)row * a.H + head) * a.col_tiles + cc / A4_COLS) * splits * REC;
  __shared__ float w[A4_MAX_SPLIT];
  __shared__ float sum, part[HD];
  const int d = threadIdx.x % HD, h = threadIdx.x / HD;
  float v[HALF];
#pragma unroll
  for (int s = 0; s < HALF; ++s)
    v[s] = 2 * s + h < splits ? rec[(size_t)(2 * s + h) * REC + c * HD + d] : 0.f;
  // a model's decode step sees its own entry at least
  bool sees = true;
  if (a.qkv == nullptr) {
    const int len = a.hdr != nullptr ? a.hdr->pos[a.row_lane[row]] + a.n_q : a.lens[row];
    sees = max(0, min(len, a.max_ctx)) - a.n_q + cc / a.group >= 0;
  }
  if (threadIdx.x < 32) {
    float m[2], l[2], M = A4_NONE, L = 0.f;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int s = threadIdx.x + 32 * u;
      m[u] = s < splits ? rec[(size_t)s * REC + A4_COLS * HD + c] : A4_NONE;
      l[u] = s < splits ? rec[(size_t)s * REC + A4_COLS * HD + A4_COLS + c] : 0.f;
      M = fmaxf(M, m[u]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const float f = exp2f(m[u] - M);
      w[threadIdx.x + 32 * u] = f;
      L = fmaf(l[u], f, L);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    if (threadIdx.x == 0) sum = L;
  }
  __syncthreads();
  float acc = 0.f;
#pragma unroll
  for (int s = 0; s < HALF; ++s)
    if (2 * s + h < splits) acc = fmaf(v[s], w[2 * s + h], acc);
  if (h == 1) part[d] = acc;
  __syncthreads();
  if (h == 0) {
    const float L = sum;
    a.out[(size_t)(row * a.n_q + cc / a.group) * a.out_stride + (size_t)(head * a.group + cc % a.group) * HD + d] =
        a4_output(acc + part[d], L, sees);
  }
}

// How the launch is cut up: CTAs per (row, cache head, column tile), their warps, the
// slots a warp takes in turn, and the records that go through the workspace.
struct A4Split {
  int ctas, warps, passes, records;
};

template <int HD>
size_t a4_smem_bytes(const A4Split& p, int cols) {
  const size_t slots = (size_t)p.warps * p.passes, c = std::min(cols, A4_COLS);
  const size_t ring = (size_t)p.warps * A4_STAGES * A4<HD>::WORDS * 4;
  const size_t records = (slots * (HD + 2) + slots / A4_GROUP * 2 + HD + 2) * c * sizeof(float);
  return p.passes > 1 ? ring + records : std::max(ring, records);
}

// The split of a caller's attention, for n (row, cache head, column tile) units.
//
// One CTA of 12 warps per SM leaves a cluster's join out, or needs one of two CTAs only;
// it takes whole SMs, of which 38 to 60 and 75 to 125 units leave many idle.  Four warps:
// four CTAs per SM; a cluster of eight for each of 74 units finds no place at once.  Heads of
// 128, us with 12 warps and with four:
//   positions  38 units      64         74         75         88         128        148
//        512   6.5   5.3   6.5  5.6   6.6  6.7   6.2  6.7   6.5  7.0   7.3  8.0   7.5  11.5
//       1024   7.8   7.0   8.7  8.2   9.0  12.2  8.9  10.1  9.2  10.5  9.5  10.7  9.7  14.3
//       2112  10.7  10.9  11.2 11.7  11.4  16.2 14.1  12.5 14.4  12.9 15.2  16.7 15.6  22.3
//       4096  15.3  14.2  16.3 15.5  16.7  20.8 23.4  17.8 23.7  20.5 25.2  25.9 25.8  32.2
//       8192  25.0  19.3  27.2 26.6  27.2  32.9 42.9  29.9 44.0  33.0 44.9  45.1 46.0  57.4
//      16384  44.2  29.9  46.1 43.3  46.8  56.4 79.8  51.8 79.8  58.6 82.1  81.4 82.8 103.5
// (heads of 64 alike).  So 12 warps where seven eighths of the SMs get a CTA; else up to 1024
// positions where a unit has one CTA, and between 1024 and 4096.
//
// More than a cluster's eight cost a second launch and a workspace: one lane of 16 heads
// takes 12.3 us in a cluster and 10.3 through the workspace at 4096 positions (12.3 and 13.3
// with two lanes), 16.4 and 13.2 at 8192.
A4Split a4_split(int max_ctx, long n) {
  const int tiles = (max_ctx + A4_TILE - 1) / A4_TILE;
  const int wide = std::min((tiles + A4_WIDE - 1) / A4_WIDE, n <= 74 ? 2 : 1);
  if (n > 37 && n <= 148 && tiles > A4_GROUP &&
      (8 * n * wide >= 7 * 148 || (tiles <= 32 ? wide == 1 : tiles < 128)))
    return {wide, A4_WIDE, 1, 0};
  const int c = (int)std::min<long>((tiles + A4_GROUP - 1) / A4_GROUP, std::max(1L, 148 * 4 / n));
  if (max_ctx < kInt4SplitCtx || c <= A4_MAX_CLUSTER) return {std::min(c, A4_MAX_CLUSTER), A4_GROUP, 1, 0};
  return {std::min(c, A4_MAX_SPLIT), A4_GROUP, 1, std::min(c, A4_MAX_SPLIT)};
}

// The split of a model's attention, whose results must not depend on how many lanes
// run: the groups of four slots, and the way they are joined, follow from max_ctx.  Where
// one CTA of 12 warps takes a unit, 75 to 125 units leave SMs idle, as above.
// Below kInt4SplitCtx six groups, in a CTA each or all in one; from there on 24,
// through the workspace.
template <int HD>
A4Split a4_lane_split(int max_ctx, long n, int cols) {
  const int tiles = (max_ctx + A4_TILE - 1) / A4_TILE;
  constexpr int wide = A4_WIDE / A4_GROUP;
  if (max_ctx < kInt4SplitCtx) {
    const int groups = std::min((tiles + A4_GROUP - 1) / A4_GROUP, 2 * wide);
    if (n > 74 && groups == 2 * wide) return {1, A4_WIDE, 2, 0};
    return {groups, A4_GROUP, 1, 0};
  }
  constexpr int groups = 8 * wide;
  if (n * groups <= 148 * 4) return {groups, A4_GROUP, 1, groups};
  A4Split p = {8, A4_WIDE, 1, groups};
  while (p.ctas > 1 && n * p.ctas > 148) {
    const A4Split q = {p.ctas / 2, A4_WIDE, p.passes * 2, groups};
    if (a4_smem_bytes<HD>(q, cols) > A4_MAX_SMEM) break;
    p = q;
  }
  return p;
}

template <int HD, int WARPS, bool FUSED>
tl_status launch_a4_kernel(const AttnInt4Args& a, const A4Split& p, size_t smem, cudaStream_t s) {
  static std::atomic<uint64_t> attr_done{0};
  TL_TRY(once_per_device(attr_done, []() -> tl_status {
    TL_CUDA(cudaFuncSetAttribute(attn_int4_kernel<HD, WARPS, FUSED>, cudaFuncAttributeMaxDynamicSharedMemorySize, A4_MAX_SMEM));
    return ok();
  }));
  const dim3 grid(p.ctas, a.H * a.col_tiles, a.n_rows);
  const cudaError_t e = launch_pdl_cluster(attn_int4_kernel<HD, WARPS, FUSED>, grid, dim3(32 * WARPS), smem, s,
                                           p.records ? 1u : (unsigned)p.ctas, a);
  if (e != cudaSuccess)
    return set_error(TL_ERR_CUDA, "launch of attn_int4_kernel failed: %s", cudaGetErrorString(e));
  return ok();
}

template <int HD, int WARPS>
tl_status launch_a4_warps(const AttnInt4Args& a, const A4Split& p, size_t smem, cudaStream_t s) {
  return a.qkv ? launch_a4_kernel<HD, WARPS, true>(a, p, smem, s) : launch_a4_kernel<HD, WARPS, false>(a, p, smem, s);
}

template <int HD>
A4Split a4_split_of(const AttnInt4Args& a, int cols) {
  const long n = (long)a.n_rows * a.H * ((cols + A4_COLS - 1) / A4_COLS);
  return a.lane_split ? a4_lane_split<HD>(a.max_ctx, n, cols) : a4_split(a.max_ctx, n);
}

template <int HD>
tl_status launch_a4(const AttnInt4Args& a0, cudaStream_t s) {
  AttnInt4Args a = a0;
  const int cols = a.n_q * a.group;
  a.col_tiles = (cols + A4_COLS - 1) / A4_COLS;
  const A4Split p = a4_split_of<HD>(a, cols);
  a.passes = p.passes;
  if (!p.records) a.ws = nullptr;
  else if (!a.ws) return set_error(TL_ERR_INVALID_ARG, "4-bit attention: a context of %d needs a workspace", a.max_ctx);
  const size_t smem = a4_smem_bytes<HD>(p, cols);
  if (p.warps == A4_WIDE) TL_TRY((launch_a4_warps<HD, A4_WIDE>(a, p, smem, s)));
  else TL_TRY((launch_a4_warps<HD, A4_GROUP>(a, p, smem, s)));
  if (p.records)
    TL_LAUNCH_PDL(attn_int4_merge_kernel<HD>, dim3(a.H * cols, a.n_rows), 2 * HD, 0, s, a, p.records);
  return ok();
}

}  // namespace

// Workspace of a call with these sizes (the arguments that set the split).
size_t attn_int4_workspace(const AttnInt4Args& a) {
  const int cols = a.n_q * a.group;
  const A4Split p = a.hd == 128 ? a4_split_of<128>(a, cols) : a4_split_of<64>(a, cols);
  return (size_t)a.n_rows * a.H * ((cols + A4_COLS - 1) / A4_COLS) * p.records * A4_COLS * (a.hd + 2) * sizeof(float);
}

tl_status launch_attn_int4(const AttnInt4Args& a, cudaStream_t s) {
  if (a.n_rows == 0) return ok();
  if (a.hd == 128) return launch_a4<128>(a, s);
  if (a.hd == 64) return launch_a4<64>(a, s);
  return set_error(TL_ERR_UNSUPPORTED, "head_dim %d not supported", a.hd);
}

}  // namespace tl
