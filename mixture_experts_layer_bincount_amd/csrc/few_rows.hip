// The experts of 17 .. 64 tokens as two weight streams.
//
//   h_r = silu(x_t W1_e^T) * (x_t W3_e^T)      for grouped row r of expert e, token t
//   y_r = h_r W2_e^T                           (the combine weighs and adds a token's)
//
// What bounds it: the touched experts' weights, as for fewer tokens, but the tokens
// no longer fit one MFMA column tile.  So the rows are grouped by expert first (the
// layer's own route and dispatch), and a segment is up to 32 rows of one expert, two
// column tiles: with one tile the Mixtral widths at 64 tokens (16 rows an expert) would
// read half the experts' weights twice.  Segments of the same expert are neighbours in
// the order of work, so what they share comes from the last-level cache.  A workgroup is
// eight waves that split an item's k range; h is kept in three bf16 terms and nothing
// is added in an order that depends on timing, as in the form for fewer tokens.  (The
// grouped GEMM kernels read the weights faster, 64 tokens of the Mixtral widths 505 us,
// but two terms of h and one accumulator over the whole of k leave an error of 2.6e-6,
// with 4-bit codes widened beside an offset 4e-5, where fp32 products leave 1.3e-6.)
#include <algorithm>

#include "moe_internal.h"
#include "weight_stream.h"

namespace moe {
namespace {

constexpr int kWaves = 8;
constexpr int kThreads = kWaves * 64;
constexpr int kTiles = 2;              // column tiles of a segment
constexpr int kRows = 16 * kTiles;     // and its rows at most
constexpr int kUp = 2;                 // gate/up item: row tiles of W1, and of W3
constexpr int kDown = 4;               // down item: row tiles of W2
constexpr int kRed = kWaves * 4 * 256; // floats: a column tile of the waves' partial sums
static_assert(2 * kUp == 4 && kDown == 4, "four row tiles an item");

struct RowsParams {
  const uint16_t* x;          // [T, d]
  const int32_t* offsets;     // [E + 1] the experts' grouped rows
  const int32_t* perm_token;  // [P_max] their tokens
  const void* W1; const void* W3; const void* W2;
  const float* s1; const float* s3; const float* s2;
  const void* W1s; const void* W3s; const void* W2s;
  const float* s1s; const float* s3s; const float* s2s;
  uint16_t* H;                // [P_max (+ T), 3, d_ff]; the shared expert's rows last
  float* Y;                   // [P_max (+ T), d]
  int64_t P_max;
  int T, d, E, d_ff, has_shared;
};

// The segments in LDS, the shared expert's first: expert (E: the shared one) | the
// segment's number within the expert << 16 | the expert's segments << 24.  Returns
// their number; called by all threads.
__device__ __forceinline__ int list_segments(const RowsParams& p, uint32_t* segs, int* sums) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = uniform(tid >> 6);
  const int shared = p.has_shared ? (p.T + kRows - 1) / kRows : 0;
  if (tid < shared) segs[tid] = (uint32_t)p.E | (uint32_t)tid << 16 | (uint32_t)shared << 24;
  const int per = (p.E + kThreads - 1) / kThreads;
  int mine = 0;
  for (int i = 0; i < per; ++i) {
    const int e = min(tid * per + i, p.E - 1);
    const int n = p.offsets[e + 1] - p.offsets[e];
    mine += tid * per + i < p.E ? (n + kRows - 1) / kRows : 0;
  }
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(incl, o, 64);
    if (lane >= o) incl += v;
  }
  if (lane == 63) sums[wave] = incl;
  __syncthreads();
  int at = shared + incl - mine, total = shared;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) at += sums[w];
    total += sums[w];
  }
  for (int i = 0; i < per; ++i) {
    const int e = min(tid * per + i, p.E - 1);
    const int n = p.offsets[e + 1] - p.offsets[e];
    const int c = tid * per + i < p.E ? (n + kRows - 1) / kRows : 0;
    for (int j = 0; j < 64 / kRows; ++j)
      if (j < c) segs[at + j] = (uint32_t)e | (uint32_t)j << 16 | (uint32_t)c << 24;
    at += c;
  }
  __syncthreads();
  return uniform(total);
}

// Work item q of nseg * tiles: a segment and a row tile.  An expert's segments take
// turns on each of its tiles.
struct RowsItem {
  int e, tile, rows;   // e = -1: the shared expert
  int64_t row0;        // first grouped row
  int first;           // first token (shared expert) or first entry of perm_token
};

__device__ __forceinline__ RowsItem rows_item(const RowsParams& p, const uint32_t* segs, int tiles,
                                              int q) {
  const int s = q / tiles;
  const uint32_t v = (uint32_t)uniform((int)segs[s]);
  const int first = s - (int)(v >> 16 & 255), count = (int)(v >> 24);
  const int in = q - first * tiles, j = in % count;
  const int e = (int)(v & 0xFFFFu);
  RowsItem it;
  it.tile = uniform(in / count);
  if (e == p.E) {
    it.e = -1;
    it.first = uniform(j * kRows);
    it.rows = uniform(min(kRows, p.T - j * kRows));
    it.row0 = p.P_max + j * kRows;
  } else {
    const int o = uniform(p.offsets[e]), end = uniform(p.offsets[e + 1]);
    it.e = e;
    it.first = uniform(o + j * kRows);
    it.rows = uniform(min(kRows, end - o - j * kRows));
    it.row0 = it.first;
  }
  return it;
}

// The waves' partial tiles of one column tile to LDS (row r of 16 x 16 tile i of wave w
// at (w * 4 + i) * 256: column-major), for everyone to add.
__device__ __forceinline__ void share_tile(float* red, int ct, const f32x4 (&acc)[4][kTiles]) {
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  __syncthreads();  // what lay there before is read
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *(f32x4*)&red[(wave * 4 + i) * 256 + r * 16 + g * 4] = acc[i][ct];
  __syncthreads();
}

__device__ __forceinline__ float add_waves(const float* red, int i) {
  float v = 0.f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) v += red[(w * 4 + i) * 256 + (threadIdx.x & 255)];
  return v;
}

// Gate/up: 32 hidden columns of a segment.
template <int WQ>
__global__ __launch_bounds__(kThreads, 2) void few_gate_up_kernel(RowsParams p) {
  extern __shared__ __align__(16) float lds[];
  constexpr int LS = StreamFmt<WQ>::LS;
  constexpr int PD = WQ == WS_BF16 ? 4 : WQ == WS_INT4 ? 1 : 2;
  float* red = lds;
  uint32_t* segs = (uint32_t*)(lds + kRed + kWaves);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = uniform(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int nseg = list_segments(p, segs, (int*)(lds + kRed));
  const int tiles = p.d_ff / (16 * kUp);
  const int64_t rowb = weight_bytes<WQ>(p.d);
  const int steps = p.d / LS;
  const StepMap<WQ> map{steps % 2 == 0 ? 1 : 0};
  const StepShare share(0, steps, wave, kWaves, map.pair, 0);
  const rsrc_t xr = buffer_of(p.x, (int64_t)p.T * p.d * 2);
  for (int q = blockIdx.x; q < nseg * tiles; q += gridDim.x) {
    const RowsItem it = rows_item(p, segs, tiles, q);
    const int f0 = it.tile * (16 * kUp);
    const int64_t moff = ((it.e < 0 ? 0 : (int64_t)it.e * p.d_ff) + f0) * rowb;
    rsrc_t wr[2 * kUp];
#pragma unroll
    for (int t = 0; t < kUp; ++t) {
      wr[2 * t] = buffer_of((const char*)(it.e < 0 ? p.W1s : p.W1) + moff + t * 16 * rowb, 16 * rowb);
      wr[2 * t + 1] =
          buffer_of((const char*)(it.e < 0 ? p.W3s : p.W3) + moff + t * 16 * rowb, 16 * rowb);
    }
    uint32_t aoff[kTiles];
#pragma unroll
    for (int ct = 0; ct < kTiles; ++ct) {
      const int c = min(ct * 16 + r, it.rows - 1);
      const int t = it.e < 0 ? it.first + c : p.perm_token[it.first + c];
      aoff[ct] = ct * 16 + r < it.rows ? (uint32_t)t * (uint32_t)p.d * 2u + map.lane_a(g) : kNowhere;
    }
    f32x4 acc[2 * kUp][kTiles];
    zero_frags(acc);
    stream_rows<WQ, 2 * kUp, kTiles, 1, PD, kLoadPlain>(
        map, wr, (uint32_t)(r * rowb) + map.lane_w(g), xr, aoff, 0u, share, acc, [] {});
    float sc1 = 1.f, sc3 = 1.f;
    if (WQ != WS_BF16) {
      const int gi = f0 / kFp8Group;
      sc1 = kWeightUnit<WQ> *
            (it.e < 0 ? p.s1s[gi] : p.s1[(int64_t)it.e * (p.d_ff / kFp8Group) + gi]);
      sc3 = kWeightUnit<WQ> *
            (it.e < 0 ? p.s3s[gi] : p.s3[(int64_t)it.e * (p.d_ff / kFp8Group) + gi]);
    }
    // entry: row tile tid / 256, row of the segment, hidden column
    const int half = tid >> 8, c = (tid >> 4) & 15;
#pragma unroll
    for (int ct = 0; ct < kTiles; ++ct) {
      share_tile(red, ct, acc);
      const float ga = sc1 * add_waves(red, 2 * half), up = sc3 * add_waves(red, 2 * half + 1);
      uint32_t hb, mb, lb;
      split3(ga / (1.f + __expf(-ga)) * up, hb, mb, lb);
      // two neighbouring columns per store, by the even lane
      const uint32_t hv = hb | (uint32_t)__shfl_xor((int)hb, 1, 64) << 16;
      const uint32_t mv = mb | (uint32_t)__shfl_xor((int)mb, 1, 64) << 16;
      const uint32_t lv = lb | (uint32_t)__shfl_xor((int)lb, 1, 64) << 16;
      if (ct * 16 + c < it.rows && !(tid & 1)) {
        uint32_t* o = (uint32_t*)(p.H + (it.row0 + ct * 16 + c) * 3 * p.d_ff + f0 + half * 16 +
                                  (tid & 15));
        o[0] = hv;
        o[p.d_ff / 2] = mv;
        o[p.d_ff] = lv;
      }
    }
  }
}

// Down: 64 output columns of a segment.
template <int WQ>
__global__ __launch_bounds__(kThreads, 2) void few_down_kernel(RowsParams p) {
  extern __shared__ __align__(16) float lds[];
  constexpr int LS = StreamFmt<WQ>::LS;
  constexpr int PD = WQ == WS_BF16 ? 3 : 1;
  float* red = lds;
  uint32_t* segs = (uint32_t*)(lds + kRed + kWaves);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = uniform(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int nseg = list_segments(p, segs, (int*)(lds + kRed));
  const int tiles = p.d / (16 * kDown);  // (d is a multiple of 64)
  const int64_t rowb = weight_bytes<WQ>(p.d_ff);
  const int steps = p.d_ff / LS;
  const StepMap<WQ> map{steps % 2 == 0 ? 1 : 0};
  for (int q = blockIdx.x; q < nseg * tiles; q += gridDim.x) {
    const RowsItem it = rows_item(p, segs, tiles, q);
    const int n0 = it.tile * (16 * kDown);
    const char* b = (const char*)(it.e < 0 ? p.W2s : p.W2) +
                    ((it.e < 0 ? 0 : (int64_t)it.e * p.d) + n0) * rowb;
    rsrc_t wr[kDown];
#pragma unroll
    for (int i = 0; i < kDown; ++i) wr[i] = buffer_of(b + i * 16 * rowb, 16 * rowb);
    uint32_t aoff[kTiles];
#pragma unroll
    for (int ct = 0; ct < kTiles; ++ct)
      aoff[ct] = ct * 16 + r < it.rows
                     ? (uint32_t)(ct * 16 + r) * 6u * (uint32_t)p.d_ff + map.lane_a(g) : kNowhere;
    const rsrc_t hr = buffer_of(p.H + it.row0 * 3 * p.d_ff, (int64_t)it.rows * 6 * p.d_ff);
    f32x4 acc[kDown][kTiles];
    zero_frags(acc);
    stream_rows<WQ, kDown, kTiles, 3, PD, kLoadPlain>(
        map, wr, (uint32_t)(r * rowb) + map.lane_w(g), hr, aoff, (uint32_t)p.d_ff * 2u,
        StepShare(0, steps, wave, kWaves, map.pair, it.tile), acc, [] {});
    float sc = 1.f;
    if (WQ != WS_BF16) {
      const int gi = n0 / kFp8Group;
      sc = kWeightUnit<WQ> * (it.e < 0 ? p.s2s[gi] : p.s2[(int64_t)it.e * (p.d / kFp8Group) + gi]);
    }
    // entries: row of the segment, output columns 16 (tid / 256 * 2 + i) + tid % 16
    const int c = (tid >> 4) & 15, i0 = (tid >> 8) * 2;
#pragma unroll
    for (int ct = 0; ct < kTiles; ++ct) {
      share_tile(red, ct, acc);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float v = sc * add_waves(red, i0 + i);
        if (ct * 16 + c < it.rows)
          p.Y[(it.row0 + ct * 16 + c) * p.d + n0 + (i0 + i) * 16 + (tid & 15)] = v;
      }
    }
  }
}

template <int WQ>
hipError_t launch(const RowsParams& p, int64_t segs, hipStream_t st) {
  const size_t lds = 4 * (kRed + kWaves + (size_t)segs);
  // (no more workgroups than the device holds at once, two a CU, or than items)
  const int64_t most = 2 * (int64_t)current_device_cus();
  const int64_t up = std::min(most, segs * (p.d_ff / (16 * kUp)));
  few_gate_up_kernel<WQ><<<(unsigned)up, kThreads, lds, st>>>(p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t down = std::min(most, segs * (p.d / (16 * kDown)));
  few_down_kernel<WQ><<<(unsigned)down, kThreads, lds, st>>>(p);
  return hipGetLastError();
}

}  // namespace

size_t few_rows_bytes(const moe_shape& s, int64_t H_rows) { return (size_t)H_rows * s.d_ff * 6; }

hipError_t launch_few_rows(const moe_shape& s, const WsLayout& L, const moe_weights& w,
                           const void* x, const int32_t* offsets, const int32_t* perm_token,
                           void* H, float* y_perm, hipStream_t st) {
  RowsParams p{};
  p.x = (const uint16_t*)x;
  p.offsets = offsets;
  p.perm_token = perm_token;
  p.W1 = w.W1; p.W3 = w.W3; p.W2 = w.W2; p.s1 = w.s1; p.s3 = w.s3; p.s2 = w.s2;
  p.W1s = w.W1s; p.W3s = w.W3s; p.W2s = w.W2s; p.s1s = w.s1s; p.s3s = w.s3s; p.s2s = w.s2s;
  p.H = (uint16_t*)H;
  p.Y = y_perm;
  p.P_max = L.P_max;
  p.T = (int)s.T; p.d = s.d; p.E = s.E; p.d_ff = s.d_ff; p.has_shared = s.has_shared ? 1 : 0;
  // sum over the experts of ceil(rows / kRows), and the shared expert's
  const int64_t A = L.P_max;
  const int64_t segs = std::min<int64_t>(s.E, A) + A / kRows +
                       (s.has_shared ? (s.T + kRows - 1) / kRows : 0);
  if (segs == 0) return hipSuccess;  // (no room for any token: every row is dropped)
  switch (s.w_dtype) {
    case MOE_DT_BF16: return launch<WS_BF16>(p, segs, st);
    case MOE_DT_FP8_E4M3: return launch<WS_FP8>(p, segs, st);
    case MOE_DT_INT8: return launch<WS_INT8>(p, segs, st);
    case MOE_DT_INT4: return launch<WS_INT4>(p, segs, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace moe
