// Streaming product of weight rows with a few activation rows on bf16 MFMA,
// shared by the few-token kernels: D[w, c] = sum_k W[w, k] a[c, k].
//
// v_mfma_f32_16x16x32_bf16 takes 16 weight rows as its A operand and 16
// activation rows (columns of D) as its B operand.  With so few columns the
// product is bound by the weights' bytes from HBM, so each weight byte is
// read once, straight into the registers the MFMA reads it from: a lane
// (r = lane & 15, g = lane >> 4) loads 16 bytes of row r per step.  Those are 8
// (bf16), 16 (8-bit) or 32 (4-bit) consecutive inputs k; the sum over k is the
// same in any order as long as the activations use the lane's own k, so no
// shuffle is needed: a step covers LS = 32, 64 or 128 inputs, LS/4 a lane, and
// feeds LS/32 MFMAs.  Steps come in pairs where a row has an even number of
// them: a lane's two loads are 32 consecutive bytes, so the four lanes of a row
// take a whole 128-byte line with two loads one after the other rather than
// half a line each.  Activations come from L2 (every workgroup reads them).
#pragma once

#include "moe_internal.h"

namespace moe {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2s __attribute__((ext_vector_type(2)));

enum { WS_BF16 = 0, WS_FP8 = 1, WS_INT8 = 2, WS_INT4 = 3 };

template <int WQ>
struct StreamFmt {
  static constexpr int LS = WQ == WS_BF16 ? 32 : WQ == WS_INT4 ? 128 : 64;  // inputs per step
  static constexpr int MF = LS / 32;                                        // MFMAs per step
};

// Bytes of n consecutive weights.
template <int WQ>
__device__ __host__ __forceinline__ constexpr int64_t weight_bytes(int64_t n) {
  return WQ == WS_BF16 ? n * 2 : WQ == WS_INT4 ? n / 2 : n;
}

// What a widened weight's unit is: int4 codes are widened to n / 16 (see widen),
// which the weights' scale makes up for, exactly.
template <int WQ>
constexpr float kWeightUnit = WQ == WS_INT4 ? 16.f : 1.f;

// Byte B of a word, sign-extended, as a float: one sub-word conversion (left
// to itself the compiler splits the word into bytes first, at twice the
// instructions and four times the registers).
template <int B>
__device__ __forceinline__ float signed_byte(uint32_t v) {
  float f;
  if constexpr (B == 0)
    asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_0"
        : "=v"(f) : "v"(v));
  else if constexpr (B == 1)
    asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_1"
        : "=v"(f) : "v"(v));
  else if constexpr (B == 2)
    asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_2"
        : "=v"(f) : "v"(v));
  else
    asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_3"
        : "=v"(f) : "v"(v));
  return f;
}

// The low four bits of byte B of a word, a signed n, as n / 16.
template <int B>
__device__ __forceinline__ float signed_nibble(uint32_t v) {
  float f;
  if constexpr (B == 0)
    asm("v_cvt_off_f32_i4_sdwa %0, %1 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_0"
        : "=v"(f) : "v"(v));
  else if constexpr (B == 1)
    asm("v_cvt_off_f32_i4_sdwa %0, %1 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_1"
        : "=v"(f) : "v"(v));
  else if constexpr (B == 2)
    asm("v_cvt_off_f32_i4_sdwa %0, %1 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_2"
        : "=v"(f) : "v"(v));
  else
    asm("v_cvt_off_f32_i4_sdwa %0, %1 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_3"
        : "=v"(f) : "v"(v));
  return f;
}

// Two values that bf16 holds exactly, packed: their upper halves.
__device__ __forceinline__ uint32_t pack_exact(float lo, float hi) {
  return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
}

// The 8 inputs of MFMA i of a loaded step as bf16, exactly (int4: n / 16).
template <int WQ>
__device__ __forceinline__ bf16x8 widen(const u32x4& q, int i) {
  if constexpr (WQ == WS_BF16) {
    return __builtin_bit_cast(bf16x8, q);
  } else if constexpr (WQ == WS_FP8) {
    // e4m3 values are all bf16 values: the scaled conversion with scale 1
    const bf16x2s p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[2 * i], 1.0f, false);
    const bf16x2s p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[2 * i], 1.0f, true);
    const bf16x2s p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[2 * i + 1], 1.0f, false);
    const bf16x2s p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[2 * i + 1], 1.0f, true);
    return bf16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
  } else if constexpr (WQ == WS_INT8) {
    bf16x8 r;  // at most 7 significant bits per code: exact
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      r[4 * h] = (__bf16)signed_byte<0>(q[2 * i + h]);
      r[4 * h + 1] = (__bf16)signed_byte<1>(q[2 * i + h]);
      r[4 * h + 2] = (__bf16)signed_byte<2>(q[2 * i + h]);
      r[4 * h + 3] = (__bf16)signed_byte<3>(q[2 * i + h]);
    }
    return r;
  } else {
    // 4-bit codes c = n + 8 (so c ^ 8 is n's two's complement), byte b of a group
    // holding input b in its low nibble and input b + 4 in its high one.  (Patterns
    // of 24 + n are made with half the instructions, but 24 times the activations'
    // sum, taken off again, leaves three times the error of the plain sum.)
    const uint32_t lo = q[i] ^ 0x88888888u, hi = lo >> 4;
    u32x4 r;
    r[0] = pack_exact(signed_nibble<0>(lo), signed_nibble<1>(lo));
    r[1] = pack_exact(signed_nibble<2>(lo), signed_nibble<3>(lo));
    r[2] = pack_exact(signed_nibble<0>(hi), signed_nibble<1>(hi));
    r[3] = pack_exact(signed_nibble<2>(hi), signed_nibble<3>(hi));
    return __builtin_bit_cast(bf16x8, r);
  }
}

// Three bf16 terms of a value (24 bits; NaN and a value past bf16's range keep
// their first term).
__device__ __forceinline__ void split3(float v, uint32_t& h, uint32_t& m, uint32_t& l) {
  h = f32_to_bf16_bits_any(v);
  float rest = v - bf16_bits_to_f32(h);
  if ((h & 0x7F80u) == 0x7F80u) rest = 0.f;
  m = f32_to_bf16_bits(rest);
  l = f32_to_bf16_bits(rest - bf16_bits_to_f32(m));
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// A raw buffer over [ptr, ptr + bytes), bytes < 2^31, from values that are the
// same in every lane.  Loads past its end return zero: that is how rows past
// a matrix' end and columns without a token (offset kNowhere) read as zeros.
typedef __amdgpu_buffer_rsrc_t rsrc_t;
constexpr uint32_t kNowhere = 0x80000000u;
__device__ __forceinline__ rsrc_t buffer_of(const void* ptr, int64_t bytes) {
  const uint64_t a = (uint64_t)ptr;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
  return __builtin_amdgcn_make_buffer_rsrc((void*)(((uint64_t)hi << 32) | lo), (short)0,
                                           __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000);
}
constexpr int kLoadPlain = 0, kLoadAgent = 16;  // cache policy: as usual, agent scope

// Where a lane's 16 bytes of step s lie in its row (`pair`: see above), and its
// first activation; lane_w and lane_a are the lane's part of the offsets.
template <int WQ>
struct StepMap {
  static constexpr int LS = StreamFmt<WQ>::LS;
  int pair;  // 0 or 1
  __device__ __forceinline__ uint32_t lane_w(int g) const { return g * (pair ? 32u : 16u); }
  __device__ __forceinline__ uint32_t lane_a(int g) const { return g * (pair ? LS : LS / 2); }
  __device__ __forceinline__ uint32_t w(int s) const {
    return pair ? (uint32_t)(s >> 1) * 128u + (s & 1) * 16u : (uint32_t)s * 64u;
  }
  // the lane's first input of step s after its first one of step 0
  __device__ __forceinline__ int input(int s) const {
    return pair ? (s >> 1) * (LS * 2) + (s & 1) * (LS / 4) : s * LS;
  }
  __device__ __forceinline__ int lane_input(int g) const { return g * (pair ? LS / 2 : LS / 4); }
  __device__ __forceinline__ uint32_t a(int s) const {
    return pair ? (uint32_t)(s >> 1) * (LS * 4) + (s & 1) * (LS / 2) : (uint32_t)s * (LS * 2);
  }
};

// A wave's share of the steps [begin, end) of a row: of every W consecutive
// pairs (or steps) one, so that the W waves of a workgroup read a row's
// consecutive lines at about the same time and DRAM pages stay open (one token,
// Mixtral widths, gate/up items by their time stamps: 6.4 TB/s, against 5.4 with a
// part of the row for each wave).
// The walk starts `turn` (a row tile's own number) into the share: row tiles
// that are streamed at the same time are whole rows apart, and at equal k many
// of their lines would lie in the same memory channels.  (The down items' rate was
// the same without it.)
struct StepShare {
  int begin, end, count, stride, pair, start;
  __device__ __forceinline__ StepShare(int b, int e, int wave, int W, int pr, int turn) {
    pair = pr;
    stride = W;
    begin = uniform(b + (pr ? 2 * wave : wave));
    end = uniform(e);
    const int groups = (e - b + (pr ? 2 * W : W) - 1) / (pr ? 2 * W : W);
    count = uniform(pr ? 2 * groups : groups);  // the same for every wave
    start = groups > 0 ? uniform(pr ? turn % groups * 2 : turn % groups) : 0;
  }
  __device__ __forceinline__ int step(int j) const {
    j += start;
    if (j >= count) j -= count;
    return pair ? begin + (j >> 1) * 2 * stride + (j & 1) : begin + j * stride;
  }
};

// acc[rt][ct] += the 16 x 16 product of row tile rt's weights and column tile
// ct's activations, over the wave's share of the rows' steps (the share's count may exceed them: those load zeros).
//   wr[rt] buffer from the row tile's first row to the end of its rows
//   wlane  the lane's byte offset: (lane & 15) * row bytes + map.lane_w
//   ar     the activations' buffer; aoff[ct] the lane's byte offset of its
//          column's row plus map.lane_a, or kNowhere; NP planes of them `plane`
//          bytes apart are summed (values held in NP bf16 terms); AUX their
//          load's cache policy
//   kleft  TAIL only (rows that may end inside a step or pair of steps): inputs of
//          the row from the lane's first one of step 0 on; what lies past them
//          counts as zero on both sides
//   ready  called once, after the first weight loads are under way and before
//          the first activation load (by every wave, with or without steps)
template <int WQ, int RT, int NCT, int NP, int PD, int AUX, bool TAIL = false, typename Ready>
__device__ __forceinline__ void stream_rows(const StepMap<WQ>& map, const rsrc_t (&wr)[RT], uint32_t wlane, rsrc_t ar,
                                            const uint32_t (&aoff)[NCT], uint32_t plane,
                                            const StepShare& share, f32x4 (&acc)[RT][NCT],
                                            Ready&& ready, int kleft = 0) {
  constexpr int MF = StreamFmt<WQ>::MF;
  const int n = share.count;  // (scalar loop control: no execution masks in the pipeline)
  u32x4 w[PD][RT];
  u32x4 a[PD][NCT][NP][MF];
  auto load_w = [&](int i, int j) __attribute__((always_inline)) {
    const int s = share.step(j);
    const bool in = s < share.end && (!TAIL || map.input(s) < kleft);
    const uint32_t o = in ? wlane + map.w(s) : kNowhere;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
      w[i][rt] = __builtin_amdgcn_raw_buffer_load_b128(wr[rt], o, 0, kLoadPlain);
  };
  auto load_a = [&](int i, int j) __attribute__((always_inline)) {
    const int s = share.step(j);
#pragma unroll
    for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
      for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int m = 0; m < MF; ++m)
          a[i][ct][p][m] = __builtin_amdgcn_raw_buffer_load_b128(
              ar,
              s < share.end && (!TAIL || map.input(s) + m * 8 < kleft)
                  ? aoff[ct] + p * plane + map.a(s) + m * 16 : kNowhere,
              0, AUX);
  };
  auto compute = [&](int i) __attribute__((always_inline)) {
#pragma unroll
    for (int m = 0; m < MF; ++m) {
      bf16x8 ww[RT];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) ww[rt] = widen<WQ>(w[i][rt], m);
#pragma unroll
      for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          const bf16x8 b = __builtin_bit_cast(bf16x8, a[i][ct][p][m]);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
            acc[rt][ct] =
                __builtin_amdgcn_mfma_f32_16x16x32_bf16(ww[rt], b, acc[rt][ct], 0, 0, 0);
        }
    }
  };
#pragma unroll
  for (int i = 0; i < PD; ++i)
    if (i < n) load_w(i, i);
  ready();
#pragma unroll
  for (int i = 0; i < PD; ++i)
    if (i < n) load_a(i, i);
  for (int j = 0; j < n; j += PD) {
#pragma unroll
    for (int i = 0; i < PD; ++i) {
      if (j + i < n) compute(i);
      if (j + i + PD < n) {
        load_w(i, j + i + PD);
        load_a(i, j + i + PD);
      }
    }
  }
}

template <int RT, int NCT>
__device__ __forceinline__ void zero_frags(f32x4 (&acc)[RT][NCT]) {
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int ct = 0; ct < NCT; ++ct) acc[rt][ct] = f32x4{0.f, 0.f, 0.f, 0.f};
}

}  // namespace
}  // namespace moe
