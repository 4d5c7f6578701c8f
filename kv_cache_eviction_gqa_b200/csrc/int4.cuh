// The 4-bit page format and what its kernels share.
//
// A page holds 16 entries (tokens) of one (sequence, kv head) unit in 20 D bytes. NG = D / 32
// groups of 32 consecutive elements, each with an fp16 scale s and zero z; an element is c s + z.
//   [ 0,  8D)  K codes, entry i at i D/2: u32 word (t, g) = t NG + g, nibble j: element 32g + 8t + j
//   [ 8D, 16D) V codes, entry i at 8D + i D/2: u16 half (r, g) = r NG + g, nibble j: element 32g + 4r + j
//   [16D, 17D) K scales [16][NG] fp16      [17D, 18D) K zeros [16][NG]
//   [18D, 19D) V scales, entry i = 8 hi + 2 t + e, group g at ((t NG + g) 2 + hi) 2 + e
//   [19D, 20D) V zeros, in the same order
// The orders are those of the m16n8k16 operands of the attention kernel: a lane (r, t) takes its
// words of a K row, its halves of a V row and its token pairs' V scales with one wide load each.
// A record is whole rows of codes and a few halves of metadata, so eviction moves it bytewise.
#pragma once
#include "qe_internal.cuh"

constexpr int kInt4Page = 16;
constexpr int kInt4Tickets = 4;   // words of the status array before the attention's tickets

// Scale and zero of a group from its exact minimum and maximum: s = fp16(f32(f32(max - min) / 15)), z =
// fp16(min). The quotient is the correctly rounded one: q0 = RN(d RN(1/15)), corrected once by its
// exact remainder (Markstein's division by a known constant; equal to IEEE division for every
// float32 significand, and what underflows is 0 in fp16 either way).
__device__ __forceinline__ uint32_t int4_meta(float mn, float mx) {
  const float d = __fsub_rn(mx, mn), r15 = 0.0666666701436042785644531f;   // RN(1/15)
  float q = __fmul_rn(d, r15);
  q = isinf(d) ? d : __fmaf_rn(__fmaf_rn(-15.f, q, d), r15, q);
  return static_cast<uint32_t>(__half_as_ushort(__float2half_rn(q))) |
         (static_cast<uint32_t>(__half_as_ushort(__float2half_rn(mn))) << 16);
}
__device__ __forceinline__ float int4_scale(uint32_t meta) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(meta & 0xffffu)));
}
__device__ __forceinline__ float int4_zero(uint32_t meta) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(meta >> 16)));
}
// 1 / (15 s), to about 2^-22; 0 for s == 0
__device__ __forceinline__ float int4_inv15(uint32_t meta) {
  const float s = int4_scale(meta);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s * 15.f));
  return s == 0.f ? 0.f : r;
}

// y = (x - z) / (15 s) saturated to [0, 1], and how far 15 y is from the integer that adding 1.5 x 2^23
// rounds it to; the sum's low bits are that integer
constexpr float kInt4Magic = 12582912.f;   // 1.5 x 2^23: bits 0x4B400000
constexpr float kInt4Near = 0.5f - 0x1p-17f;
__device__ __forceinline__ float int4_round(float x, float z, float inv15, float* off) {
  const float y = __saturatef(__fmul_rn(__fsub_rn(x, z), inv15));   // NaN gives 0
  const float t = __fmaf_rn(y, 15.f, kInt4Magic);
  *off = __fmaf_rn(y, 15.f, __fsub_rn(kInt4Magic, t));
  return t;
}
// The codes n of four elements with those next to a half-integer decided by correctly rounded division;
// out of line (elements of few bits do fall on half-integers: 7 in 10 000 of normal bf16 values, so
// every tenth warp comes here)
static __device__ __noinline__ uint32_t int4_codes_near(float a, float b, float c, float d, uint32_t meta, float inv15,
                                                        uint32_t n) {
  const float s = int4_scale(meta), z = int4_zero(meta);
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
    const float x = i == 0 ? a : i == 1 ? b : i == 2 ? c : d;
    float off;
    int4_round(x, z, inv15, &off);
    if (fabsf(off) > kInt4Near)   // negative quotients convert to 0
      n = (n & ~(15u << (4 * i))) | min(__float2uint_rn(__fdiv_rn(__fsub_rn(x, z), s)), 15u) << (4 * i);
  }
  return n;
}
// Codes of four elements, nibble by nibble: clamp(rint(f32(f32(x - z) / s)), 0, 15), 0 if s == 0, ties
// to even. The clamp's bounds are integers, so it may come first; 15 y is within 4e-6 of the quotient,
// and within 2^-17 of a half-integer the division decides, so the codes are the definition's in every case.
__device__ __forceinline__ uint32_t int4_codes(float a, float b, float c, float d, uint32_t meta, float inv15) {
  const float z = int4_zero(meta), x[4] = {a, b, c, d};
  float off[4];
  uint32_t n = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i)   // the constant's low 16 bits are 0
    n += __float_as_uint(int4_round(x[i], z, inv15, &off[i])) << (4 * i);
  n &= 0xffffu;
  const float far = fmaxf(fmaxf(fabsf(off[0]), fabsf(off[1])), fmaxf(fabsf(off[2]), fabsf(off[3])));
  return far > kInt4Near ? int4_codes_near(a, b, c, d, meta, inv15, n) : n;
}

// device view of a qe_int4_cache
struct Int4View {
  uint8_t* pages;
  int32_t* table;      // [U][max_pages]
  int32_t* lengths;    // [U]
  int32_t* seen;       // [B]
  float* mass;         // [n_pages][16]
  int32_t* pos;        // [n_pages][16]
  int32_t* status;     // code, detail, append's ticket, -, then attend's tickets
  int B, Hkv, max_pages, n_pages;
};

// host: argument checks of a cache and its view (QE_OK or an error)
int int4_view(const qe_int4_cache* c, Int4View* v);
