// One step of decode attention over the 4-bit cache, with the weights that its entries collect.
//
// Per unit (sequence b, kv head) with G query heads and entries i of length L:
//   p_hi = softmax_i(q_h . k_i / sqrt(D)),  out_h = sum_i p_hi v_i,  mass_i += sum_h p_hi,
// k and v being the values c s + z that the entries stand for. Each page is read once; the codes
// go to the warp-level tensor cores (m16n8k16) as they are, never expanded to c s + z:
//   masking a word with 0x000F000F (0x00F000F0) leaves two codes as the fp16 subnormals
//   c 2^-24 (c 2^-20), exact operands; so with tokens as MMA rows and the heads as columns
//     scores   s_ih = sum_g s_ig (c_ig . q_hg) + z_ig (sum of q_h over g):  one accumulator a group,
//              scaled by its row's s_ig in float32, and one m16n8k8 for all zeros (the sum of q
//              over a group split into two fp16 parts);
//     output   O_dh = sum_i c_id (s_ig p_ih) + sum_i z_ig p_ih:  the scale goes onto the weights.
// q is scaled per head by a power of two into fp16's range. The weights are rounded to fp16 (times
// 16, times s once more): 2^-11 relative, below the output's own rounding in bf16 and equal to it
// in fp16; their sums, the maxima and the scores are float32.
//
// Split: the pages of all units form one flat list, cut into equal ranges, one a CTA, so batches of
// very different lengths load every SM alike. Warp w of a CTA takes every 4th page of a range,
// each page one bulk copy into the warp's own ring. A range may cross units: per (CTA, unit) piece
// the warps merge in shared memory and leave one partial (m, l, O). The scores of a weighing call go
// to scratch (float32, mostly L2) and the second kernel turns them into weights once the unit's
// maximum and sum are known.
#include <math.h>

#include "int4.cuh"
#include "warp_mma.cuh"

namespace {

constexpr int kWarps = 4;
constexpr int kStages = 4;
constexpr int kCtasPerSm = 4;
constexpr int kMinPages = 8;        // pages of a range below which more CTAs only add merging
constexpr int kCombinePages = 64;   // pages of a unit that a CTA of the second kernel weighs

struct AttendArgs {
  Int4View c;
  const void* q;        // [B][Hq][D] rows at q_stride
  long long q_stride;
  void* out;            // [B][Hq][D] dtype
  int Hq, G, GP, weigh; // GP: G rounded up to a pair
  float cs;             // log2(e) / sqrt(D)
  int max_ctas;
  int32_t* prefix;      // [U + 1] pages before each unit, then the number of CTAs that took part
  float* part_ml;       // [slots][2][8]
  float* part_o;        // [slots][8][D]
  float* scores;        // [flat pages][16][GP], log2 domain
};

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t movm_t(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  uint32_t y;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
  return y;
}
__device__ __forceinline__ float h_lo(uint32_t w) { return __half2float(__ushort_as_half((unsigned short)(w & 0xffffu))); }
__device__ __forceinline__ float h_hi(uint32_t w) { return __half2float(__ushort_as_half((unsigned short)(w >> 16))); }

__device__ __forceinline__ void mma_k16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  MmaOp<__half>::run(c, a0, a1, a2, a3, b0, b1);
}
__device__ __forceinline__ void mma_k8(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5}, {%6}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(b0));
}

// pages of unit u, 0 for a length out of range (recorded)
__device__ __forceinline__ int unit_pages(const Int4View& c, int u) {
  const int len = c.lengths[u];
  if (len < 0 || (long long)len > (long long)c.max_pages * kInt4Page) {
    qe_record_error(c.status, QE_ERR_INVALID_ARG, u);
    return 0;
  }
  return (len + kInt4Page - 1) / kInt4Page;
}

// first flat page of CTA c's range: floor(c P / C)
__device__ __forceinline__ int range_at(int c, int P, int C) { return (int)((long long)c * P / C); }
// the CTA whose range holds flat page p
__device__ __forceinline__ int cta_of(int p, int P, int C) { return (int)((((long long)p + 1) * C - 1) / P); }
__device__ __forceinline__ int ctas_for(int P, int most) {
  const int c = (P + kMinPages - 1) / kMinPages;
  return c < most ? c : most;
}

template <int D>
struct AttendLayout {
  static constexpr int PAGE = 20 * D;
  static constexpr int RING = kStages * PAGE;            // a warp's; also holds its O for the merge
  static constexpr int SMEM = kWarps * RING + kWarps * kStages * 8;
  static_assert(RING >= 8 * D * 4, "a warp's partial output fits its ring");
};

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm) int4_attend_kernel(AttendArgs a) {
  using L = AttendLayout<D>;
  constexpr int NG = D / 32;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_total, s_unit, s_base;
  __shared__ float s_m[kWarps][8], s_l[kWarps][8], s_z[kWarps][8][NG];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, t = lane & 3;
  const Int4View& c = a.c;
  const int U = c.B * c.Hkv;
  uint8_t* ring = smem + warp * L::RING;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kWarps * L::RING) + warp * kStages;
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&bars[s], 1);
    fence_mbar_init();
  }
  // ---- this CTA's range of the flat page list ----
  if (warp == 0) {
    int total = 0;
    for (int u0 = 0; u0 < U; u0 += 32) {
      const int n = u0 + lane < U ? unit_pages(c, u0 + lane) : 0;
      int inc = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      if (blockIdx.x == 0 && u0 + lane < U) a.prefix[u0 + lane] = total + inc - n;
      total += __shfl_sync(0xffffffffu, inc, 31);
    }
    const int C = ctas_for(total, a.max_ctas);
    if (blockIdx.x == 0 && lane == 0) a.prefix[U] = total;
    if (lane == 0) s_total = total;
    if ((int)blockIdx.x < C) {           // the unit that holds the range's first page
      const int p = range_at(blockIdx.x, total, C);
      int before = 0;
      for (int u0 = 0; u0 < U; u0 += 32) {
        const int n = u0 + lane < U ? unit_pages(c, u0 + lane) : 0;
        int inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += y;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, before + inc > p);
        if (past) {
          const int w = __ffs(past) - 1;
          if (lane == w) s_unit = u0 + w, s_base = before + inc - n;
          break;
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
      }
    }
  }
  __syncthreads();
  const int P = s_total, C = ctas_for(P, a.max_ctas), cta = blockIdx.x;
  if (cta >= C) return;
  const int p_end = range_at(cta + 1, P, C);
  int p = range_at(cta, P, C), u = s_unit, base = s_base;
  uint32_t fills = 0;                    // copies this warp has waited for: stage and phase
  bool ok = true;

  while (p < p_end) {
    // ---- one piece: pages p .. p1 - 1 of unit u ----
    int np = unit_pages(c, u);
    while (np == 0 || p >= base + np) {  // skip empty units
      base += np;
      np = unit_pages(c, ++u);
    }
    const int p1 = min(p_end, base + np), len = c.lengths[u];
    const int b = u / c.Hkv, kvh = u % c.Hkv;
    const int32_t* table = c.table + (size_t)u * c.max_pages - base;
    const int mine = (p1 - p - warp + kWarps - 1) / kWarps;   // this warp's pages: p + warp + kWarps i
    auto issue = [&](int i) {
      const int page = table[p + warp + kWarps * i];
      const int s = (fills + i) % kStages;
      if (page < 0 || page >= c.n_pages) {  // nothing is read: the page counts as masked
        qe_record_error(c.status, QE_ERR_DEVICE_FAULT, u);
        mbar_arrive_expect_tx(&bars[s], 0);
        return;
      }
      mbar_arrive_expect_tx(&bars[s], L::PAGE);
      bulk_g2s(ring + s * L::PAGE, c.pages + (size_t)page * L::PAGE, L::PAGE, &bars[s]);
    };
    if (lane == 0)
      for (int i = 0; i < min(mine, kStages); ++i) issue(i);

    // ---- the queries: fp16 fragments scaled by 2^e, and their sums over groups ----
    uint32_t qf[2 * NG][2];
    uint32_t qs;
    float k1[2], k2[2];                  // accumulators to log2 scores, for heads 2t and 2t + 1
    {
      float x[NG][8];
      float mx = 0.f;
      if (r < a.G) {
        const T* src = static_cast<const T*>(a.q) + b * a.q_stride + (kvh * a.G + r) * D + 8 * t;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const uint4 w = *reinterpret_cast<const uint4*>(src + 32 * g);
          x[g][0] = Elem<T>::lo(w.x), x[g][1] = Elem<T>::hi(w.x), x[g][2] = Elem<T>::lo(w.y), x[g][3] = Elem<T>::hi(w.y);
          x[g][4] = Elem<T>::lo(w.z), x[g][5] = Elem<T>::hi(w.z), x[g][6] = Elem<T>::lo(w.w), x[g][7] = Elem<T>::hi(w.w);
#pragma unroll
          for (int j = 0; j < 8; ++j) mx = fmaxf(mx, fabsf(x[g][j]));
        }
      } else {
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
          for (int j = 0; j < 8; ++j) x[g][j] = 0.f;
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      // the largest element lands in [2^13, 2^14): exponents -100..60 keep every factor finite
      const int e = max(-100, min(60, 13 - ((int)(__float_as_uint(mx) >> 23) - 127)));
      const float f = __uint_as_float((uint32_t)(e + 127) << 23);
      float sum[NG];
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        sum[g] = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          x[g][j] *= f;
          sum[g] += x[g][j];
        }
        sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 1);
        sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 2);
        sum[g] *= 0.0625f;
        // nibbles 1, 3, 5, 7 arrive as 16 c: their queries are divided by 16
        qf[2 * g][0] = pack_h2(x[g][0], x[g][4]);
        qf[2 * g][1] = pack_h2(x[g][1] * 0.0625f, x[g][5] * 0.0625f);
        qf[2 * g + 1][0] = pack_h2(x[g][2], x[g][6]);
        qf[2 * g + 1][1] = pack_h2(x[g][3] * 0.0625f, x[g][7] * 0.0625f);
      }
      // rows of the 8 x 8 operand: the groups' sums, then what rounding them to fp16 left
      const int g0 = NG == 4 ? 2 * (t & 1) : 0;
      const float u0 = NG == 4 && g0 ? sum[NG - 2] : sum[0], u1 = NG == 4 && g0 ? sum[NG - 1] : sum[1];
      const uint32_t hi = pack_h2(u0, u1), lo = pack_h2(u0 - h_lo(hi), u1 - h_hi(hi));
      qs = NG == 4 ? (t < 2 ? hi : lo) : (t == 0 ? hi : t == 1 ? lo : 0u);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int eh = __shfl_sync(0xffffffffu, e, (2 * t + j) * 4);
        k1[j] = a.cs * __uint_as_float((uint32_t)(24 - eh + 127) << 23);
        k2[j] = a.cs * __uint_as_float((uint32_t)(4 - eh + 127) << 23);
      }
    }
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;   // heads 2t, 2t + 1
    float o[2 * NG][4], oz[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int x = 0; x < 2 * NG; ++x)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[x][j] = 0.f;

    for (int i = 0; i < mine; ++i) {
      const uint32_t f = fills + i;
      const int s = f % kStages;
      const int fp = p + warp + kWarps * i;
      ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(&bars[s], (f / kStages) & 1, c.status, 6001));
      if (!ok) break;
      const uint8_t* pg = ring + s * L::PAGE;
      // ---- scores ----
      float sc[4] = {0.f, 0.f, 0.f, 0.f}, sz[4] = {0.f, 0.f, 0.f, 0.f};
      {
        uint32_t ka[2][NG], ks[2][NG / 2];
#pragma unroll
        for (int hr = 0; hr < 2; ++hr) {
          const uint8_t* row = pg + (r + 8 * hr) * (D / 2) + t * (NG * 4);
          const uint8_t* meta = pg + 16 * D + (r + 8 * hr) * (NG * 2);
          if (NG == 4) {
            const uint4 w = *reinterpret_cast<const uint4*>(row);
            ka[hr][0] = w.x, ka[hr][1] = w.y, ka[hr][NG - 2] = w.z, ka[hr][NG - 1] = w.w;
            const uint2 m = *reinterpret_cast<const uint2*>(meta);
            ks[hr][0] = m.x, ks[hr][NG / 2 - 1] = m.y;
          } else {
            const uint2 w = *reinterpret_cast<const uint2*>(row);
            ka[hr][0] = w.x, ka[hr][1] = w.y;
            ks[hr][0] = *reinterpret_cast<const uint32_t*>(meta);
          }
        }
        const int zo = NG == 4 ? (t & 1) * 4 : 0;
        mma_k8(sz, *reinterpret_cast<const uint32_t*>(pg + 17 * D + r * (NG * 2) + zo),
               *reinterpret_cast<const uint32_t*>(pg + 17 * D + (r + 8) * (NG * 2) + zo), qs);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          float acc[4] = {0.f, 0.f, 0.f, 0.f};
          const uint32_t x0 = ka[0][g], x1 = ka[1][g], y0 = x0 >> 8, y1 = x1 >> 8;
          mma_k16(acc, x0 & 0x000f000fu, x1 & 0x000f000fu, x0 & 0x00f000f0u, x1 & 0x00f000f0u, qf[2 * g][0], qf[2 * g][1]);
          mma_k16(acc, y0 & 0x000f000fu, y1 & 0x000f000fu, y0 & 0x00f000f0u, y1 & 0x00f000f0u, qf[2 * g + 1][0],
                  qf[2 * g + 1][1]);
          const float s0 = g & 1 ? h_hi(ks[0][g / 2]) : h_lo(ks[0][g / 2]);
          const float s1 = g & 1 ? h_hi(ks[1][g / 2]) : h_lo(ks[1][g / 2]);
          sc[0] = fmaf(acc[0], s0, sc[0]), sc[1] = fmaf(acc[1], s0, sc[1]);
          sc[2] = fmaf(acc[2], s1, sc[2]), sc[3] = fmaf(acc[3], s1, sc[3]);
        }
        sc[0] = fmaf(sc[0], k1[0], sz[0] * k2[0]), sc[1] = fmaf(sc[1], k1[1], sz[1] * k2[1]);
        sc[2] = fmaf(sc[2], k1[0], sz[2] * k2[0]), sc[3] = fmaf(sc[3], k1[1], sz[3] * k2[1]);
      }
      // entries of this page inside the unit; none when its table entry was out of range
      const int pgid = table[fp];
      const int live = pgid < 0 || pgid >= c.n_pages ? 0 : min(kInt4Page, len - (fp - base) * kInt4Page);
      if (live < kInt4Page) {
        if (r >= live) sc[0] = sc[1] = -INFINITY;
        if (r + 8 >= live) sc[2] = sc[3] = -INFINITY;
      }
      if (a.weigh && 2 * t < a.GP) {
        float* dst = a.scores + ((size_t)fp * kInt4Page + r) * a.GP + 2 * t;
        *reinterpret_cast<float2*>(dst) = make_float2(sc[0], sc[1]);
        *reinterpret_cast<float2*>(dst + 8 * a.GP) = make_float2(sc[2], sc[3]);
      }
      // ---- softmax: the maxima move rarely, and then all lanes of a head together ----
      const float x0 = fmaxf(sc[0], sc[2]), x1 = fmaxf(sc[1], sc[3]);
      if (__any_sync(0xffffffffu, x0 > m0 || x1 > m1)) {
        float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) {
          n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, w));
          n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, w));
        }
        const float f0 = m0 == n0 ? 1.f : ex2f(m0 - n0), f1 = m1 == n1 ? 1.f : ex2f(m1 - n1);
        m0 = n0, m1 = n1;
        l0 *= f0, l1 *= f1;
#pragma unroll
        for (int x = 0; x < 2 * NG; ++x) o[x][0] *= f0, o[x][1] *= f1, o[x][2] *= f0, o[x][3] *= f1;
        oz[0] *= f0, oz[1] *= f1;
      }
      // 16 p: the factor cancels in the output and keeps p s clear of fp16's subnormals
      const float b0f = m0 == -INFINITY ? 0.f : m0 - 4.f, b1f = m1 == -INFINITY ? 0.f : m1 - 4.f;
      const float p00 = ex2f(sc[0] - b0f), p01 = ex2f(sc[1] - b1f), p10 = ex2f(sc[2] - b0f), p11 = ex2f(sc[3] - b1f);
      l0 += p00 + p10, l1 += p01 + p11;
      const uint32_t pb0 = movm_t(pack_h2(p00, p01)), pb1 = movm_t(pack_h2(p10, p11));
      // ---- output: rows are elements, the contraction runs over the 16 entries ----
      uint32_t vs[NG][2], vz[2];
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const uint2 w = *reinterpret_cast<const uint2*>(pg + 18 * D + (t * NG + g) * 8);
        vs[g][0] = w.x, vs[g][1] = w.y;
      }
      {
        const uint2 w = *reinterpret_cast<const uint2*>(pg + 19 * D + (t * NG + (r & (NG - 1))) * 8);
        vz[0] = r < NG ? w.x : 0u, vz[1] = r < NG ? w.y : 0u;
      }
      if (live < kInt4Page) {            // what dead slots hold may be anything: 0 x NaN is not 0
        auto keep = [&](int i0) { return (i0 < live ? 0xffffu : 0u) | (i0 + 1 < live ? 0xffff0000u : 0u); };
        const uint32_t k_lo = keep(2 * t), k_hi = keep(2 * t + 8);
#pragma unroll
        for (int g = 0; g < NG; ++g) vs[g][0] &= k_lo, vs[g][1] &= k_hi;
        vz[0] &= k_lo, vz[1] &= k_hi;
      }
      mma_k16(oz, vz[0], 0u, vz[1], 0u, pb0, pb1);
      uint32_t va[4][NG / 2];            // entries 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint8_t* row = pg + 8 * D + (2 * t + (j & 1) + 8 * (j >> 1)) * (D / 2) + r * (NG * 2);
        if (NG == 4) {
          const uint2 w = *reinterpret_cast<const uint2*>(row);
          va[j][0] = w.x, va[j][NG / 2 - 1] = w.y;
        } else {
          va[j][0] = *reinterpret_cast<const uint32_t*>(row);
        }
      }
      __syncwarp();
      if (lane == 0 && i + kStages < mine) issue(i + kStages);   // every lane has read the page
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const uint32_t sel = g & 1 ? 0x7632u : 0x5410u;
        const uint32_t lo = __byte_perm(va[0][g / 2], va[1][g / 2], sel), hi = __byte_perm(va[2][g / 2], va[3][g / 2], sel);
        const uint32_t q0 = hmul2(pb0, vs[g][0]), q1 = hmul2(pb1, vs[g][1]);
        mma_k16(o[2 * g], lo & 0x000f000fu, lo & 0x00f000f0u, hi & 0x000f000fu, hi & 0x00f000f0u, q0, q1);
        mma_k16(o[2 * g + 1], (lo >> 8) & 0x000f000fu, (lo >> 8) & 0x00f000f0u, (hi >> 8) & 0x000f000fu,
                (hi >> 8) & 0x00f000f0u, q0, q1);
      }
    }
    fills += mine > 0 ? mine : 0;
    if (!ok) break;                      // the status word holds the reason

    // ---- merge the warps ----
#pragma unroll
    for (int w = 4; w < 32; w <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, w);
      l1 += __shfl_xor_sync(0xffffffffu, l1, w);
    }
    __syncwarp();
    if (r == 0) s_m[warp][2 * t] = m0, s_m[warp][2 * t + 1] = m1, s_l[warp][2 * t] = l0, s_l[warp][2 * t + 1] = l1;
    if (r < NG) s_z[warp][2 * t][r] = oz[0], s_z[warp][2 * t + 1][r] = oz[1];
    float* wo = reinterpret_cast<float*>(ring);
    constexpr float kLo = 16777216.f, kHi = 1048576.f;   // 2^24, 2^20
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        *reinterpret_cast<float4*>(wo + (2 * t + j) * D + 32 * g + 4 * r) =
            make_float4(o[2 * g][j] * kLo, o[2 * g][j + 2] * kHi, o[2 * g + 1][j] * kLo, o[2 * g + 1][j + 2] * kHi);
    __syncthreads();
    {
      const size_t slot = (size_t)cta + u;
      for (int x = tid; x < a.G * D; x += kWarps * 32) {
        const int h = x / D, d = x % D;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][h]);
        float acc = 0.f, l = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float f = s_m[w][h] == -INFINITY ? 0.f : ex2f(s_m[w][h] - M);
          acc = fmaf(f, reinterpret_cast<const float*>(smem + w * L::RING)[h * D + d] + s_z[w][h][d / 32], acc);
          l = fmaf(f, s_l[w][h], l);
        }
        a.part_o[slot * 8 * D + x] = acc;
        if (d == 0) a.part_ml[slot * 16 + h] = M, a.part_ml[slot * 16 + 8 + h] = l;
      }
    }
    fence_proxy_async_smem();            // the rings take bulk copies again
    __syncthreads();
    p = p1;
  }
}

// Joins a unit's partials: chunk 0 writes the output, and every chunk adds its entries' weights.
template <typename T, int D>
__global__ void __launch_bounds__(128) int4_combine_kernel(AttendArgs a) {
  __shared__ float s_M[8], s_il[8];
  const Int4View& c = a.c;
  const int U = c.B * c.Hkv, u = blockIdx.y, chunk = blockIdx.x, tid = threadIdx.x;
  const int base = a.prefix[u], P = a.prefix[U], np = a.prefix[u + 1] - base;
  const int b = u / c.Hkv, kvh = u % c.Hkv;
  if (chunk * kCombinePages >= np) {
    if (chunk == 0) {                    // no entries: the output is 0
      T* dst = static_cast<T*>(a.out) + ((size_t)b * a.Hq + kvh * a.G) * D;
      for (int x = tid; x < a.G * D; x += 128) dst[x] = Elem<T>::from_f(0.f);
    }
    return;
  }
  const int C = ctas_for(P, a.max_ctas);
  const int c0 = cta_of(base, P, C), c1 = cta_of(base + np - 1, P, C);
  if (tid < a.G) {
    float M = -INFINITY, l = 0.f;
    for (int x = c0; x <= c1; ++x) M = fmaxf(M, a.part_ml[((size_t)x + u) * 16 + tid]);
    for (int x = c0; x <= c1; ++x) {
      const float m = a.part_ml[((size_t)x + u) * 16 + tid];
      if (m != -INFINITY) l = fmaf(a.part_ml[((size_t)x + u) * 16 + 8 + tid], ex2f(m - M), l);
    }
    s_M[tid] = M;
    s_il[tid] = l > 0.f ? 1.f / l : 0.f;
  }
  __syncthreads();
  if (chunk == 0) {
    T* dst = static_cast<T*>(a.out) + ((size_t)b * a.Hq + kvh * a.G) * D;
    for (int x = tid; x < a.G * D; x += 128) {
      const int h = x / D;
      float acc = 0.f;
      for (int y = c0; y <= c1; ++y) {
        const float m = a.part_ml[((size_t)y + u) * 16 + h];
        if (m != -INFINITY) acc = fmaf(a.part_o[((size_t)y + u) * 8 * D + x], ex2f(m - s_M[h]), acc);
      }
      dst[x] = Elem<T>::from_f(acc * s_il[h]);
    }
  }
  if (!a.weigh) return;
  const int len = c.lengths[u];
  const int e1 = min(len, (chunk + 1) * kCombinePages * kInt4Page);
  for (int e = chunk * kCombinePages * kInt4Page + tid; e < e1; e += 128) {
    const int page = c.table[(size_t)u * c.max_pages + e / kInt4Page];
    if (page < 0 || page >= c.n_pages) continue;   // recorded by the first kernel
    const float* sc = a.scores + ((size_t)base * kInt4Page + e) * a.GP;
    float w = 0.f;
    for (int h = 0; h < a.G; ++h) w += ex2f(sc[h] - s_M[h] + 4.f) * s_il[h];
    c.mass[(size_t)page * kInt4Page + e % kInt4Page] += w;
  }
}

struct ScratchLayout {
  size_t prefix, part_ml, part_o, scores, bytes;
  ScratchLayout(long long units, int G, int D, long long max_pages, int ctas) {
    auto r = [](size_t x) { return (x + 255) & ~size_t(255); };
    const size_t slots = (size_t)ctas + units;
    prefix = 0;
    part_ml = r((units + 1) * 4);
    part_o = part_ml + r(slots * 16 * 4);
    scores = part_o + r(slots * 8 * D * 4);
    bytes = scores + r((size_t)units * max_pages * kInt4Page * ((G + 1) & ~1) * 4);
  }
};

// One resident wave, whatever the device: a CTA more would only wait for another's end.
constexpr int kMaxCtas = 148 * kCtasPerSm;

template <typename T, int D>
int launch(const AttendArgs& a, cudaStream_t st) {
  using L = AttendLayout<D>;
  auto kern = int4_attend_kernel<T, D>;
  static QeOnce once;
  int dev = 0;
  const int e = qe_once_per_device(once, &dev, [&](int) {
    QE_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM));
    return QE_OK;
  });
  if (e) return e;
  const int U = a.c.B * a.c.Hkv;
  const long long most = ((long long)U * a.c.max_pages + kMinPages - 1) / kMinPages;
  kern<<<(int)(most < a.max_ctas ? most : a.max_ctas), kWarps * 32, L::SMEM, st>>>(a);
  const int chunks = a.weigh ? (a.c.max_pages + kCombinePages - 1) / kCombinePages : 1;
  int4_combine_kernel<T, D><<<dim3(chunks, U), 128, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? QE_OK : QE_ERR_CUDA;
}

}  // namespace

QE_API size_t qe_int4_scratch_bytes(int B, int Hq, int Hkv, int D, int max_pages) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || Hq / Hkv > QE_MAX_G || max_pages < 1 || (D != 64 && D != 128)) return 0;
  if ((long long)B * Hkv * max_pages * kInt4Page >= (1ll << 31)) return 0;
  return ScratchLayout((long long)B * Hkv, Hq / Hkv, D, max_pages, kMaxCtas).bytes;
}

QE_API int qe_int4_attend(const qe_int4_cache* cache, const void* q, long long q_stride, int Hq, int dtype,
                          int accumulate, void* out, void* scratch, size_t scratch_bytes, qe_stream_t stream) {
  AttendArgs a{};
  const int e = int4_view(cache, &a.c);
  if (e) return e;
  const int D = cache->D;
  if (Hq < 1 || Hq % a.c.Hkv || (dtype != QE_FP16 && dtype != QE_BF16)) return QE_ERR_INVALID_ARG;
  if (Hq / a.c.Hkv > QE_MAX_G || a.c.B * (long long)a.c.Hkv > 65535) return QE_ERR_UNSUPPORTED_SHAPE;
  if (!q || !out || !scratch || !qe_aligned(q, 16) || q_stride % 8 || q_stride < (long long)Hq * D ||
      !qe_aligned(scratch, 256))
    return QE_ERR_INVALID_ARG;
  const ScratchLayout S((long long)a.c.B * a.c.Hkv, Hq / a.c.Hkv, D, a.c.max_pages, kMaxCtas);
  if (scratch_bytes < S.bytes) return QE_ERR_WORKSPACE;
  uint8_t* w = static_cast<uint8_t*>(scratch);
  a.q = q;
  a.q_stride = q_stride;
  a.out = out;
  a.Hq = Hq;
  a.G = Hq / a.c.Hkv;
  a.GP = (a.G + 1) & ~1;
  a.weigh = accumulate != 0;
  a.cs = 1.4426950408889634f / sqrtf((float)D);
  a.max_ctas = kMaxCtas;
  a.prefix = reinterpret_cast<int32_t*>(w + S.prefix);
  a.part_ml = reinterpret_cast<float*>(w + S.part_ml);
  a.part_o = reinterpret_cast<float*>(w + S.part_o);
  a.scores = reinterpret_cast<float*>(w + S.scores);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (D == 128)
    return dtype == QE_BF16 ? launch<__nv_bfloat16, 128>(a, st) : launch<__half, 128>(a, st);
  return dtype == QE_BF16 ? launch<__nv_bfloat16, 64>(a, st) : launch<__half, 64>(a, st);
}
