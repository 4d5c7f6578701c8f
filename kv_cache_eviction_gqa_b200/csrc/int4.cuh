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

// Scale and zero of a group from its exact minimum and maximum: s = fp16(f32(f32(max - min) / 15)),
// z = fp16(min), and the code of an element: clamp(rint(f32(f32(x - z) / s)), 0, 15), 0 if s == 0,
// ties to even. The quotient is first taken with an approximate reciprocal (error below 15 x 2^-22);
// within 1e-3 of a half-integer the correctly rounded division decides, so the code is that of the
// definition in every case.
struct Int4Group {
  __half sh, zh;
  float s, z, rs;
  __device__ __forceinline__ Int4Group(float mn, float mx) {
    sh = __float2half_rn(__fdiv_rn(__fsub_rn(mx, mn), 15.f));
    zh = __float2half_rn(mn);
    s = __half2float(sh);
    z = __half2float(zh);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(rs) : "f"(s));
    if (s == 0.f) rs = 0.f;
  }
  __device__ __forceinline__ uint32_t code(float x) const {
    const float d = __fsub_rn(x, z);
    float q = __fmul_rn(d, rs);
    if (fabsf(q - rintf(q)) > 0.499f) q = __fdiv_rn(d, s);
    return min(__float2uint_rn(q), 15u);   // negative values and NaN convert to 0
  }
};

// device view of a qe_int4_cache
struct Int4View {
  uint8_t* pages;
  int32_t* table;      // [U][max_pages]
  int32_t* lengths;    // [U]
  int32_t* seen;       // [B]
  float* mass;         // [n_pages][16]
  int32_t* pos;        // [n_pages][16]
  int32_t* status;     // [4]: code, detail, append's ticket, -
  int B, Hkv, max_pages, n_pages;
};

// host: argument checks of a cache and its view (QE_OK or an error)
int int4_view(const qe_int4_cache* c, Int4View* v);
