// Low-rank adapters of many requests beside a shared projection.
//
//   y_t = base_t + bias + x_t W^T + s_a ((x_t A_a^T) B_a^T),  a = adapter_idx[t]
//
// (a row whose index lies outside [0, n) has no adapter).  Two launches:
//
//   to 64 rows   adapter_rows_kernel: S_t = s_a x_t A_a^T by some workgroups and
//                x W^T by the others, streamed into MFMA registers, d_in split over
//                the waves and over workgroups: fp32 parts; then
//                adapter_join_kernel adds them, S B^T (fp32 dot products), bias and
//                base
//   more rows    adapter_tile_kernel<PART>: S by some workgroups, 128 x 128 tiles of
//                x W^T through LDS, d_in split over workgroups, by the others; then
//                adapter_expand_kernel: the parts, S B^T on MFMA, bias and base
//   many tiles   adapter_shrink_kernel: S; then adapter_tile_kernel: 256 x 256
//                tiles whose epilogue adds S B^T, adapter by adapter
//   no W         adapter_shrink_kernel, then the join or expand kernel
//
// No sorting by adapter: the rows of a batch come in runs (prompts) or one by
// one (decode), and a 16-row tile of the shrink product simply visits the
// adapters that its rows name (each once), whose A has to be read in any case.
// From 65 rows on, blocks of 32 rows pass over all the adapters they name, too, so
// many rows of many adapters in no order cost a pass for each (4096 rows, 64 adapters
// of rank 16, 4096 -> 4096: 341 us against 157 where the rows come in runs, of rank
// 128 1600 against 293): there a batch sorted by adapter is the faster one.
// S is never rounded to fewer than 24 bits.
#include <algorithm>

#include "moe_internal.h"
#include "weight_stream.h"

namespace moe {
namespace {

constexpr int kWaves = 8;
constexpr int kThreads = kWaves * 64;
constexpr int kMaxParts = 8;   // of x W^T
constexpr int kMaxShrink = 4;  // of S

struct AdapterParams {
  const uint16_t* x;       // [T, d_in]
  const void* W;           // [d_out, d_in] or NULL
  const float* s;          // [d_out / 128]
  const float* bias;       // [d_out] or NULL
  const uint16_t* A;       // [n, R, d_in]
  const uint16_t* B;       // [n, d_out, R]
  const int32_t* ranks;    // [n] or NULL
  const float* scales;     // [n]
  const int32_t* idx;      // [T]
  const void* base;        // [T, d_out] in y's type, or NULL
  void* y;                 // [T, d_out]
  float* S;                // [KS, T, R]: S is the sum of the KS parts
  int64_t T;
  int d_in, d_out, n, R, y_f32;
  int KS, Z;       // shrink: workgroups that split d_in, and that share a row tile's adapters
  float* part;     // [KW, T, d_out]: x W^T is the sum of the KW parts
  int KW;
  int s_ranks;     // shrink: rank tiles
  int s_blocks;    // and workgroups
};

__device__ __forceinline__ int adapter_rank(const AdapterParams& p, int a) {
  return p.ranks ? max(0, min(p.ranks[a], p.R)) : p.R;
}

// ---------------------------------------------------------------- shrink
// One 16-row tile of x against 16 rows of every adapter that the tile's rows
// name (each once); Z workgroups take the adapters in turn, KS of them split
// d_in, their waves split it further.  Bound by the latency of reading the
// adapters: the launch picks Z and KS so that even one row's adapter is read by
// several workgroups.
template <int NW>
__device__ __forceinline__ void shrink_tile(const AdapterParams& p, int b, float* red) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = uniform(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  // row tiles go round fastest, z slowest: where rows come in runs only z = 0 has
  // work, which is to lie on all XCDs (4096 rows: 35 us against 17)
  const int tiles = (int)((p.T + 15) / 16);
  const int64_t t0 = (int64_t)(b % tiles) * 16;
  b /= tiles;
  const int r0 = b % p.s_ranks * 16;
  b /= p.s_ranks;
  const int ks = b % p.KS, z = b / p.KS;
  const int rows = (int)min((int64_t)16, p.T - t0);
  int mine = r < rows ? p.idx[t0 + r] : -1;  // this lane's column's adapter
  if (mine < 0 || mine >= p.n) mine = -1;
  const int all = (p.d_in + 63) / 64;  // pairs of steps
  const StepMap<WS_BF16> map{1};
  const StepShare share(all * ks / p.KS * 2, all * (ks + 1) / p.KS * 2, wave, NW, 1, 0);
  const int64_t rowb = (int64_t)p.d_in * 2;
  const rsrc_t xr = buffer_of(p.x + t0 * p.d_in, rows * rowb);
  // the element whose sum this thread finishes (the first 256 threads)
  const int col = tid >> 4;
  const int own = __shfl(mine, col & 15, 64);
  uint32_t todo = (uint32_t)__ballot(mine >= 0) & 0xFFFFu;
  for (int turn = 0; todo; ++turn) {
    const int a = __builtin_amdgcn_readlane(mine, __builtin_ctz(todo));
    todo &= ~(uint32_t)__ballot(mine == a);
    if (turn % p.Z != z) continue;
    const int rank = adapter_rank(p, a);
    const float scale = p.scales[a];
    const rsrc_t wr[1] = {
        buffer_of(p.A + ((int64_t)a * p.R + r0) * p.d_in, min(16, p.R - r0) * rowb)};
    const uint32_t aoff[1] = {mine == a ? (uint32_t)(r * rowb) + map.lane_a(g) : kNowhere};
    f32x4 acc[1][1];
    zero_frags(acc);
    stream_rows<WS_BF16, 1, 1, 1, 6, kLoadPlain, true>(
        map, wr, (uint32_t)(r * rowb) + map.lane_w(g), xr, aoff, 0u, share, acc, [] {},
        p.d_in - map.lane_input(g));
    __syncthreads();  // the previous adapter's sums are read
    *(f32x4*)&red[wave * 256 + r * 16 + g * 4] = acc[0][0];
    __syncthreads();
    const int row = r0 + (tid & 15);
    if (wave < 4 && own == a && row < p.R) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) v += red[w * 256 + tid];
      p.S[(ks * p.T + t0 + col) * p.R + row] = row < rank ? v * scale : 0.f;
    }
  }
}

__global__ __launch_bounds__(kThreads) void adapter_shrink_kernel(AdapterParams p) {
  __shared__ __align__(16) float red[kWaves * 256];
  shrink_tile<kWaves>(p, blockIdx.x, red);
}

// base + bias + v of element (t, n), rounded once to y's type.
__device__ __forceinline__ void store_y(const AdapterParams& p, int64_t t, int n, float v) {
  const int64_t o = t * p.d_out + n;
  if (p.bias) v += p.bias[n];
  if (p.y_f32) {
    if (p.base) v += ((const float*)p.base)[o];
    ((float*)p.y)[o] = v;
  } else {
    if (p.base) v += bf16_bits_to_f32(((const uint16_t*)p.base)[o]);
    ((__bf16*)p.y)[o] = (__bf16)v;
  }
}

// ---------------------------------------------------------------- rows
// The first workgroups run the shrink product, the others x W^T: 16 * RT rows of W
// against 16 * NCT rows of x, one of KW ranges of d_in, which the waves split
// further.  Bound by W's bytes (few rows of x) or by the loads of x from L2.
template <int WQ, int RT, int NCT, int PD>
__global__ __launch_bounds__(kThreads, 2) void adapter_rows_kernel(AdapterParams p) {
  constexpr int LS = StreamFmt<WQ>::LS, N = 16 * RT, kPad = 256 + 16;
  __shared__ __align__(16) float red[kWaves * RT * kPad];
  int b = blockIdx.x;
  if (b < p.s_blocks) {
    shrink_tile<kWaves>(p, b, red);
    return;
  }
  b -= p.s_blocks;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = uniform(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int tiles_n = (p.d_out + N - 1) / N;
  const int n0 = b % tiles_n * N;
  b /= tiles_n;
  const int kw = b % p.KW;
  const int64_t t0 = (int64_t)(b / p.KW) * 16 * NCT;
  const int rows = (int)min((int64_t)16 * NCT, p.T - t0);
  f32x4 acc[RT][NCT];
  zero_frags(acc);
  const int64_t rowb = weight_bytes<WQ>(p.d_in);
  // bf16: a lane's two loads of a pair of steps take whole lines; of the narrower
  // weights' longer steps the activations' lines would be the scattered ones
  constexpr int P = WQ == WS_BF16 ? 1 : 0, U = LS << P;
  const int all = (p.d_in + U - 1) / U;
  const StepMap<WQ> map{P};
  rsrc_t wr[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
    wr[i] = buffer_of((const char*)p.W + (int64_t)(n0 + i * 16) * rowb,
                      max(0, min(16, p.d_out - n0 - i * 16)) * rowb);
  uint32_t aoff[NCT];
#pragma unroll
  for (int ct = 0; ct < NCT; ++ct)
    aoff[ct] = ct * 16 + r < rows
                   ? (uint32_t)(ct * 16 + r) * (uint32_t)p.d_in * 2u + map.lane_a(g) : kNowhere;
  stream_rows<WQ, RT, NCT, 1, PD, kLoadPlain, true>(
      map, wr, (uint32_t)(r * rowb) + map.lane_w(g),
      buffer_of(p.x + t0 * p.d_in, (int64_t)rows * p.d_in * 2), aoff, 0u,
      StepShare((all * kw / p.KW) << P, (all * (kw + 1) / p.KW) << P, wave, kWaves, P, n0 / N),
      acc, [] {}, p.d_in - map.lane_input(g));
  // the waves' sums, 16 rows of x at a time; a thread keeps its output n
  const int nl = tid % N, n = n0 + nl;
  float scale = 1.f;
  if (WQ != WS_BF16) scale = kWeightUnit<WQ> * p.s[min(n, p.d_out - 1) / kFp8Group];
  float* out = p.part + ((int64_t)kw * p.T + t0) * p.d_out + n;
#pragma unroll
  for (int ct = 0; ct < NCT; ++ct) {
    if (ct) __syncthreads();
#pragma unroll
    for (int i = 0; i < RT; ++i)
      *(f32x4*)&red[(wave * RT + i) * kPad + r * 16 + g * 4] = acc[i][ct];
    __syncthreads();
#pragma unroll
    for (int h = 0; h < (RT + 1) / 2; ++h) {
      const int c = tid / N + h * (kThreads / N), col = ct * 16 + c;
      if (c >= 16 || col >= rows || n >= p.d_out) continue;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) v += red[(w * RT + nl / 16) * kPad + c * 16 + nl % 16];
      out[(int64_t)col * p.d_out] = v * scale;
    }
  }
}

// The sum of the KW parts of x W^T's element o.
__device__ __forceinline__ float sum_parts(const AdapterParams& p, int64_t o) {
  float v[kMaxParts];
#pragma unroll
  for (int i = 0; i < kMaxParts; ++i)
    v[i] = i < p.KW ? p.part[i * p.T * p.d_out + o] : 0.f;
#pragma unroll
  for (int i = 1; i < kMaxParts; ++i) v[0] += v[i];
  return v[0];
}

// One row's 128 outputs: the parts, S B^T, bias and base.  Bound by latency: all
// loads are under way before the first is used.
constexpr int kJoin = 128;
__global__ __launch_bounds__(kJoin) void adapter_join_kernel(AdapterParams p) {
  __shared__ float sv[MOE_ADAPTER_MAX_RANK];
  const int tid = threadIdx.x, n = blockIdx.x * kJoin + tid;
  const int64_t t = blockIdx.y;
  const int a = p.idx[t];
  const bool has = a >= 0 && a < p.n;
  const int rank = has ? adapter_rank(p, a) : 0;
  const int nc = min(n, p.d_out - 1);
  float s[kMaxShrink];
#pragma unroll
  for (int i = 0; i < kMaxShrink; ++i)
    s[i] = i < p.KS && tid < rank ? p.S[(i * p.T + t) * p.R + tid] : 0.f;
  float v = sum_parts(p, t * p.d_out + nc);
  const uint16_t* bp = p.B + ((int64_t)(has ? a : 0) * p.d_out + nc) * p.R;
#pragma unroll
  for (int i = 1; i < kMaxShrink; ++i) s[0] += s[i];
  if (tid < p.R) sv[tid] = s[0];
  __syncthreads();
  for (int k0 = 0; k0 < rank; k0 += 64) {
    u32x4 b[8];
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (k0 + c * 8 < rank) b[c] = *(const u32x4*)(bp + k0 + c * 8);  // (R is a multiple of 8)
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      if (k0 + c * 8 >= rank) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float bv = bf16_bits_to_f32((j & 1) ? b[c][j / 2] >> 16 : b[c][j / 2] & 0xFFFFu);
        // (what lies past the rank is not taken as a number)
        v += k0 + c * 8 + j < rank ? sv[k0 + c * 8 + j] * bv : 0.f;
      }
    }
  }
  if (n < p.d_out) store_y(p, t, n, v);
}

// ---------------------------------------------------------------- tiles
// BM rows of x by BM rows of W, k in steps of 32 through four LDS stages; BM / 32
// waves of BM / 2 x 64 (BM / 64 x 2 MFMA tiles of 32 x 32 x 16).  Two steps and more
// are on their way by LDS DMA (quantised weights through registers, widened
// exactly) while one is multiplied, and half a step's fragments are read while the
// half before it is multiplied.  What bounds it: of 540 us at 4096 rows, 4096 ->
// 14336, the DMA's share of LDS and L2 costs 85 (452 without it) and the adapters 30;
// two stages of 64 read at the start of a step took 543.  Rows are 64 bytes; 16-byte
// chunk c of row r lies at c ^ (r / 4 % 4), so the 16 rows that are read together
// lie in different banks.
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;
constexpr int kStepK = 32, kStages = 4;

// acc += S B^T of 32 rows and 32 * J outputs from n0 on, straight from L2 into MFMA
// registers (v_mfma_f32_32x32x16_bf16, register q of a lane: row (q / 4) * 8 +
// (lane / 32) * 4 + q % 4, output lane % 32), adapter by adapter of the 32 rows;
// each 16 of k run three times, over the three bf16 terms of S (the sum of its
// KS <= NK parts).  t, mine: the lane's row and its adapter or -1.  A row takes the
// sums of its own adapter only: what another's holds does not reach it, not even
// as NaN times zero.
template <int J, int NK>
__device__ __forceinline__ void add_adapters(const AdapterParams& p, int64_t t, int mine, int n0,
                                             f32x16 (&acc)[J]) {
  const int lane = threadIdx.x & 63, fr = lane & 31, fg = lane >> 5;
  uint32_t todo = (uint32_t)__ballot(mine >= 0);
  while (todo) {
    const int a = __builtin_amdgcn_readlane(mine, __builtin_ctz(todo));
    const uint32_t mask = (uint32_t)__ballot(mine == a);
    todo &= ~mask;
    const int rank = adapter_rank(p, a);
    const rsrc_t br = buffer_of(p.B + ((int64_t)a * p.d_out + n0) * p.R,
                                (int64_t)max(0, min(32 * J, p.d_out - n0)) * p.R * 2);
    f32x16 part[J];
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) part[j][q] = 0.f;
    for (int k0 = 0; k0 < rank; k0 += 16) {
      const int k = k0 + fg * 8;
      const bool in = k < rank;  // (R and k are multiples of 8)
      u32x4 bv[J];
#pragma unroll
      for (int j = 0; j < J; ++j)
        bv[j] = __builtin_amdgcn_raw_buffer_load_b128(
            br, in ? (uint32_t)((j * 32 + fr) * p.R + k) * 2u : kNowhere, 0, kLoadPlain);
      f32x4 s[NK][2];
      const float* sp = p.S + t * p.R + k;
#pragma unroll
      for (int i = 0; i < NK; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          s[i][h] = in && mine == a && (NK == 1 || i < p.KS)
                        ? *(const f32x4*)(sp + i * p.T * p.R + h * 4) : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 1; i < NK; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) s[0][h] += s[i][h];
      u32x4 term[3];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t lo[3], hi[3];
        split3(s[0][w / 2][w % 2 * 2], lo[0], lo[1], lo[2]);
        split3(s[0][w / 2][w % 2 * 2 + 1], hi[0], hi[1], hi[2]);
#pragma unroll
        for (int i = 0; i < 3; ++i) term[i][w] = lo[i] | hi[i] << 16;
#pragma unroll
        for (int j = 0; j < J; ++j) {  // past the rank: zeros, whatever B holds there
          if (k + w * 2 >= rank) bv[j][w] = 0u;
          else if (k + w * 2 + 1 >= rank) bv[j][w] &= 0xFFFFu;
        }
      }
#pragma unroll
      for (int i = 0; i < 3; ++i)
#pragma unroll
        for (int j = 0; j < J; ++j)
          part[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
              __builtin_bit_cast(bf16x8, term[i]), __builtin_bit_cast(bf16x8, bv[j]), part[j], 0,
              0, 0);
    }
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const bool own = mask >> ((q / 4) * 8 + fg * 4 + q % 4) & 1u;
#pragma unroll
      for (int j = 0; j < J; ++j) acc[j][q] += own ? part[j][q] : 0.f;
    }
  }
}

// acc += 32 rows x 32 * J outputs from n0 on of each of NB row-major [rows, d_out]
// buffers of `size`-byte values (4: fp32, 2: bf16), eight loads of each under way at
// a time; rows and outputs past the end read as zeros.
template <int J, int NB>
__device__ __forceinline__ void add_block(const AdapterParams& p, const rsrc_t (&r)[NB], int size,
                                          int n0, f32x16 (&acc)[J]) {
  const int lane = threadIdx.x & 63, fr = lane & 31, fg = lane >> 5;
#pragma unroll
  for (int h = 0; h < 2 * J; ++h) {
    const int j = h / 2, n = n0 + j * 32 + fr;
    uint32_t v[NB][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int q = h % 2 * 8 + i;
      const uint32_t m = (q / 4) * 8 + fg * 4 + q % 4;
      const uint32_t o = n < p.d_out ? (m * p.d_out + n) * (uint32_t)size : kNowhere;
#pragma unroll
      for (int k = 0; k < NB; ++k)
        v[k][i] = size == 4 ? __builtin_amdgcn_raw_buffer_load_b32(r[k], o, 0, 0)
                            : (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(r[k], o, 0, 0) << 16;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int k = 0; k < NB; ++k) acc[j][h % 2 * 8 + i] += __uint_as_float(v[k][i]);
    __builtin_amdgcn_sched_barrier(0);  // (no more values in registers at a time)
  }
}

// y of 32 rows (from t0 on, `rows` of them there) and 32 * J outputs from n0 on: bias
// and base are added, one rounding to y's type.
template <int J>
__device__ __forceinline__ void store_block(const AdapterParams& p, int64_t t0, int rows, int n0,
                                            f32x16 (&acc)[J]) {
  const int lane = threadIdx.x & 63, fr = lane & 31, fg = lane >> 5;
  const int64_t o0 = t0 * p.d_out;
  const int64_t left = (int64_t)max(0, min(32, rows)) * p.d_out;
  if (p.bias) {
#pragma unroll
    for (int j = 0; j < J; ++j) acc[j] += p.bias[min(n0 + j * 32 + fr, p.d_out - 1)];
  }
  if (p.base) {
    const int size = p.y_f32 ? 4 : 2;
    const rsrc_t br[1] = {buffer_of((const char*)p.base + o0 * size, left * size)};
    if (p.y_f32) add_block(p, br, 4, n0, acc);
    else add_block(p, br, 2, n0, acc);
  }
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const int m = (q / 4) * 8 + fg * 4 + q % 4, n = n0 + j * 32 + fr;
      if (m >= rows || n >= p.d_out) continue;
      const int64_t o = o0 + (int64_t)m * p.d_out + n;
      if (p.y_f32) ((float*)p.y)[o] = acc[j][q];
      else ((__bf16*)p.y)[o] = (__bf16)acc[j][q];
    }
}

// PART: the last workgroups run the shrink product (first, the many that find no
// adapter of their own held up the tiles: 333 rows 60 us against 46), the
// others write the fp32 parts of KW ranges of d_in; else S is there and the
// workgroup finishes its tile.
template <int WQ, int BM, bool PART>
__global__ __launch_bounds__(BM * 2, 2) void adapter_tile_kernel(AdapterParams p) {
  extern __shared__ __align__(16) char lds[];
  constexpr int kRow = kStepK * 2, kStage = 2 * BM * kRow;  // x tile, then W tile
  constexpr int NI = BM / 64;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = uniform(tid >> 6);
  int nblk = gridDim.x;
  if constexpr (PART) {
    nblk -= p.s_blocks;
    if ((int)blockIdx.x >= nblk) {
      shrink_tile<BM / 32>(p, blockIdx.x - nblk, (float*)lds);
      return;
    }
  }
  // the workgroups of one XCD (consecutive ones go round the XCDs) take
  // neighbouring tiles: eight row tiles by consecutive weight tiles
  const int tiles_n = (p.d_out + BM - 1) / BM;
  const int tiles_t = (int)((p.T + BM - 1) / BM);
  const int per = nblk / 8, rest = nblk % 8, xcd = blockIdx.x % 8;
  int b = xcd * per + min(xcd, rest) + blockIdx.x / 8;
  int kw = 0;
  if constexpr (PART) {
    kw = b / (tiles_n * tiles_t);
    b %= tiles_n * tiles_t;
  }
  const int bt = b / (8 * tiles_n) * 8;
  const int in_band = min(8, tiles_t - bt), bi = b % (8 * tiles_n);
  const int64_t t0 = (int64_t)(bt + bi % in_band) * BM;
  const int n0 = bi / in_band * BM;
  const int rows = (int)min((int64_t)BM, p.T - t0);
  const int64_t rowb = weight_bytes<WQ>(p.d_in);
  const rsrc_t xr = buffer_of(p.x + t0 * p.d_in, (int64_t)rows * p.d_in * 2);
  const rsrc_t wr = buffer_of((const char*)p.W + n0 * rowb,
                              (int64_t)min(BM, p.d_out - n0) * rowb);
  // wave (wt, wn): rows wt * BM / 2 .., weight rows wn * 64 ..
  const int wt = wave & 1, wn = wave >> 1;
  f32x16 acc[NI][2];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.f;
  // DMA: one instruction of a wave fills 16 rows (1 KiB), lane l the slot l % 4 of
  // row l / 4; wave w fills rows 32 w .. + 31.  Of quantised weights a thread loads
  // 16 bytes of a step.
  constexpr bool kDmaW = WQ == WS_BF16;
  constexpr int kLoads = kDmaW ? 4 : 3;  // of a wave and step
  const int dc = (lane & 3) ^ (lane >> 4);
  const int drow = wave * 32 + (lane >> 2);
  const uint32_t xoff = (uint32_t)drow * (uint32_t)p.d_in * 2u + dc * 16u;
  const uint32_t woff = (uint32_t)drow * (uint32_t)rowb + dc * 16u;
  const int all = (p.d_in + kStepK - 1) / kStepK;
  const int s0 = PART ? all * kw / p.KW : 0;
  const int n = (PART ? all * (kw + 1) / p.KW : all) - s0;  // > 0
  u32x4 rw[2];
  auto load = [&](int s) __attribute__((always_inline)) {
    const int k = (s0 + s) * kStepK;
    char* xt = lds + s % kStages * kStage + wave * (32 * kRow);
    const bool in = k + dc * 8 < p.d_in;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          xr, (lds_ptr_t)(xt + i * 1024), 16,
          in ? xoff + (uint32_t)i * 32u * (uint32_t)p.d_in + k * 2u : kNowhere, 0, 0, 0);
    if constexpr (kDmaW) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            wr, (lds_ptr_t)(xt + BM * kRow + i * 1024), 16,
            in ? woff + (uint32_t)i * 16u * (uint32_t)rowb + k * 2u : kNowhere, 0, 0, 0);
    } else if constexpr (WQ == WS_INT4) {
      rw[s & 1] = __builtin_amdgcn_raw_buffer_load_b128(
          wr, tid < BM ? (uint32_t)(tid * rowb) + k / 2 : kNowhere, 0, kLoadPlain);
    } else {
      rw[s & 1] = __builtin_amdgcn_raw_buffer_load_b128(
          wr, (uint32_t)((tid >> 1) * rowb) + k + (tid & 1) * 16, 0, kLoadPlain);
    }
  };
  auto put_chunk = [&](char* tile, int row, int c, bf16x8 v) __attribute__((always_inline)) {
    *(bf16x8*)(tile + row * kRow + ((c ^ (row >> 2 & 3)) << 4)) = v;
  };
  auto stage = [&](int s) __attribute__((always_inline)) {
    char* wtile = lds + s % kStages * kStage + BM * kRow;
    if constexpr (WQ == WS_INT4) {
      if (tid < BM) {
#pragma unroll
        for (int m = 0; m < 4; ++m) put_chunk(wtile, tid, m, widen<WQ>(rw[s & 1], m));
      }
    } else if constexpr (!kDmaW) {
#pragma unroll
      for (int m = 0; m < 2; ++m)
        put_chunk(wtile, tid >> 1, (tid & 1) * 2 + m, widen<WQ>(rw[s & 1], m));
    }
  };
  // this wave's transfers of all but the `later` last steps and its LDS writes are
  // done, then everyone's
  auto join = [&](int later) __attribute__((always_inline)) {
    if (later >= 2) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(2 * kLoads) : "memory");
    else if (later == 1) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kLoads) : "memory");
    else asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  const int fr = lane & 31, fg = lane >> 5;
  // fragments of half a step (16 of k)
  bf16x8 fx[2][NI], fw[2][2];
  auto read = [&](int s, int kk) __attribute__((always_inline)) {
    const char* xt = lds + s % kStages * kStage;
    const char* wtile = xt + BM * kRow;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int row = wn * 64 + j * 32 + fr;
      fw[kk][j] = *(const bf16x8*)(wtile + row * kRow + (((kk * 2 + fg) ^ (row >> 2 & 3)) << 4));
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int row = wt * (BM / 2) + i * 32 + fr;
      fx[kk][i] = *(const bf16x8*)(xt + row * kRow + (((kk * 2 + fg) ^ (row >> 2 & 3)) << 4));
    }
  };
  auto multiply = [&](int kk) __attribute__((always_inline)) {
    __builtin_amdgcn_sched_barrier(0);  // (the next half's reads go first)
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        acc[i][j] =
            __builtin_amdgcn_mfma_f32_32x32x16_bf16(fx[kk][i], fw[kk][j], acc[i][j], 0, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
  };
  // Each half's fragments are read while the half before it is multiplied: the
  // barrier that gives step s + 1 (and frees step s - 1's stage) lies between the
  // halves of step s.
  load(0);
  if (n > 1) load(1);
  stage(0);
  if (n > 2) load(2);
  join(min(n - 1, 2));
  read(0, 0);
  for (int s = 0; s < n; s += kStages) {
#pragma unroll
    for (int u = 0; u < kStages; ++u) {  // (s is a multiple of four: stages by constants)
      if (s + u >= n) break;
      if (s + u + 1 < n) stage(s + u + 1);
      read(s + u, 1);
      multiply(0);
      if (s + u + 1 < n) {
        join(min(n - 2 - s - u, 1));
        if (s + u + 3 < n) load(s + u + 3);
        read(s + u + 1, 0);
      }
      multiply(1);
    }
  }
  if constexpr (WQ != WS_BF16) {  // the weights' scales, before the adapters' part is added
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int n = n0 + wn * 64 + j * 32 + fr;
      const float sc = n < p.d_out ? kWeightUnit<WQ> * p.s[n / kFp8Group] : 0.f;
#pragma unroll
      for (int i = 0; i < NI; ++i) acc[i][j] *= sc;
    }
  }
  if constexpr (PART) {
    float* out = p.part + ((int64_t)kw * p.T + t0) * p.d_out;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const int m = wt * (BM / 2) + i * 32 + (q / 4) * 8 + fg * 4 + q % 4;
          const int n = n0 + wn * 64 + j * 32 + fr;
          if (m < rows && n < p.d_out) out[(int64_t)m * p.d_out + n] = acc[i][j][q];
        }
  } else {
    int mine[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int row = wt * (BM / 2) + i * 32 + fr;
      mine[i] = row < rows ? p.idx[t0 + row] : -1;
      if (mine[i] >= p.n) mine[i] = -1;
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int r0 = wt * (BM / 2) + i * 32;
      add_adapters<2, 1>(p, t0 + r0 + fr, mine[i], n0 + wn * 64, acc[i]);
      store_block(p, t0 + r0, rows - r0, n0 + wn * 64, acc[i]);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// The parts (if any), S B^T, bias and base of many rows: 32 rows x 32 outputs a
// wave.  Bound by reading base and the parts and writing y; of few tiles by
// latency (blocks of 64 outputs a wave and one part's loads at a time: 333 rows of
// 1416 outputs, seven parts, 28 us against 12).
constexpr int kExpandThreads = 256;
__global__ __launch_bounds__(kExpandThreads) void adapter_expand_kernel(AdapterParams p) {
  const int fr = threadIdx.x & 31;
  const int n0 = blockIdx.x * 128 + uniform(threadIdx.x >> 6) * 32;
  const int64_t t0 = (int64_t)blockIdx.y * 32;
  const int rows = (int)min((int64_t)32, p.T - t0);
  const int a = fr < rows ? p.idx[t0 + fr] : -1;
  f32x16 acc[1];
#pragma unroll
  for (int q = 0; q < 16; ++q) acc[0][q] = 0.f;
  for (int kw = 0; kw < p.KW; kw += 4) {
    rsrc_t pr[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      pr[k] = buffer_of(p.part + ((int64_t)(kw + k) * p.T + t0) * p.d_out,
                        kw + k < p.KW ? (int64_t)rows * p.d_out * 4 : 0);
    add_block(p, pr, 4, n0, acc);
  }
  add_adapters<1, kMaxShrink>(p, t0 + fr, a >= 0 && a < p.n ? a : -1, n0, acc);
  store_block(p, t0, rows, n0, acc);
}

// How a call is run.
struct Plan {
  int BM;          // tile kernel of BM x BM tiles; 0: rows kernel
  bool expand;     // joined by the expand kernel (else the join kernel)
  int RT, NCT;     // rows kernel: its tile
  int KW, KS, Z;   // KW > 0: parts
  int s_ranks, s_blocks;
};

int64_t tiles_of(const moe_adapter_shape& s, int bt, int bn) {
  return ((s.T + bt - 1) / bt) * ((s.d_out + bn - 1) / bn);
}

Plan plan_of(const moe_adapter_shape& s, bool has_w) {
  Plan q{};
  q.expand = s.T > 64;
  q.NCT = s.T <= 16 ? 1 : s.T <= 32 ? 2 : 4;
  q.RT = q.NCT;
  int64_t kw = 0;
  if (!has_w) {
  } else if (s.T <= 64) {
    // (64 rows, 4096 -> 14336, fp8: 56 us against 71 in 128 x 128 tiles; 333 rows: 53
    // against 27.)  As many row tiles of W as of x: 27 rows: 27 us with two against 30
    // with one and 28 with four; 64 rows: 49 with four against 66 with two; one row:
    // 17 with one against 19 with two.  d_in is split for two workgroups on each CU,
    // each wave with two pairs of steps or more.
    kw = std::min<int64_t>(512 / tiles_of(s, 16 * q.NCT, 16 * q.RT), s.d_in / (128 * kWaves));
    q.KW = (int)std::max<int64_t>(1, std::min<int64_t>(kMaxParts, kw));
  } else if (s.T > 256 && tiles_of(s, 256, 256) >= 150) {
    // 256 x 256 tiles when there are enough of them to keep most CUs busy, one a CU
    // (4096 inputs, bf16: 168 tiles 138 us against 161 in 128 x 128 tiles with parts,
    // 128 tiles 134 against 119, 64 tiles 131 against 75)
    q.BM = 256;
  } else {
    // two workgroups fit on a CU; d_in is split as far as that takes
    q.BM = 128;
    kw = std::min<int64_t>(512 / tiles_of(s, 128, 128), s.d_in / (8 * kStepK));
    q.KW = (int)std::max<int64_t>(1, std::min<int64_t>(kMaxParts, kw));
  }
  // the shrink product: up to 16 workgroups (with tiles, where they hold much LDS and
  // rows come in runs, 4) for the adapters of a row tile, and d_in split as long as
  // they stay few: those without an adapter of their own cost their start (27 rows,
  // 48 adapters of rank 64: 26.6 us with 1024 workgroups against 21.9 with 512; 333
  // rows in runs: 44 with 16 for a row tile against 33 with 4)
  q.s_ranks = (s.rank + 15) / 16;
  const int64_t base = ((s.T + 15) / 16) * q.s_ranks;
  q.Z = (int)std::max<int64_t>(
      1, std::min<int64_t>(std::min<int64_t>(q.expand ? 4 : 16, s.T), 1024 / base));
  kw = std::min<int64_t>(q.expand ? 256 / base : 512 / (base * q.Z), s.d_in / (64 * kWaves));
  q.KS = (int)std::max<int64_t>(1, std::min<int64_t>(q.BM == 256 ? 1 : kMaxShrink, kw));
  q.s_blocks = (int)(base * q.Z * q.KS);
  return q;
}

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

size_t s_bytes(const moe_adapter_shape& s, const Plan& q) {
  return align256((size_t)s.T * s.rank * 4 * q.KS);
}

template <int WQ, int RT, int NCT, int PD>
void launch_rows(const AdapterParams& p, hipStream_t st) {
  const int64_t blocks = p.s_blocks +
                         ((p.d_out + 16 * RT - 1) / (16 * RT)) * p.KW *
                             ((p.T + 16 * NCT - 1) / (16 * NCT));
  adapter_rows_kernel<WQ, RT, NCT, PD><<<(unsigned)blocks, kThreads, 0, st>>>(p);
}

template <int WQ, int BM, bool PART>
hipError_t launch_tile(const AdapterParams& p, hipStream_t st) {
  constexpr int lds = kStages * 2 * BM * kStepK * 2;
  const hipError_t e = hipFuncSetAttribute((const void*)adapter_tile_kernel<WQ, BM, PART>,
                                           hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (e != hipSuccess) return e;
  int64_t blocks = ((p.T + BM - 1) / BM) * ((p.d_out + BM - 1) / BM);
  if (PART) blocks = blocks * p.KW + p.s_blocks;
  adapter_tile_kernel<WQ, BM, PART><<<(unsigned)blocks, BM * 2, lds, st>>>(p);
  return hipGetLastError();
}

template <int WQ>
hipError_t launch_main(const AdapterParams& p, const Plan& q, hipStream_t st) {
  if (q.BM == 256) return launch_tile<WQ, 256, false>(p, st);
  if (q.BM == 128) return launch_tile<WQ, 128, true>(p, st);
  constexpr int PD = WQ == WS_BF16 ? 4 : WQ == WS_INT4 ? 1 : 2;
  if (q.NCT == 1) launch_rows<WQ, 1, 1, 2 * PD>(p, st);
  else if (q.NCT == 2) launch_rows<WQ, 2, 2, PD>(p, st);
  else launch_rows<WQ, 4, 4, (PD + 1) / 2>(p, st);
  return hipGetLastError();
}

hipError_t launch_weights(const moe_adapter_shape& s, const AdapterParams& p, const Plan& q,
                          hipStream_t st) {
  switch (s.w_dtype) {
    case MOE_DT_BF16: return launch_main<WS_BF16>(p, q, st);
    case MOE_DT_FP8_E4M3: return launch_main<WS_FP8>(p, q, st);
    case MOE_DT_INT8: return launch_main<WS_INT8>(p, q, st);
    case MOE_DT_INT4: return launch_main<WS_INT4>(p, q, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace

// The most that any batch of 1 .. s.T rows takes: few rows' products are cut into parts
// that many rows' are not, and a workspace made for the largest batch is to serve them
// all.  From 16 rows on a plan changes only between multiples of 16; once W takes the
// 256 x 256 tiles (no parts) and S is in one part, more rows just have more of S.
size_t adapter_workspace_bytes(const moe_adapter_shape& shape) {
  moe_adapter_shape s = shape;
  size_t most = 0;
  for (int64_t T = 1; T < shape.T + 16; T += T < 16 ? 1 : 16) {
    s.T = std::min(T, shape.T);
    const Plan q = plan_of(s, true), bare = plan_of(s, false);
    most = std::max({most, s_bytes(s, q) + (size_t)q.KW * s.T * s.d_out * 4, s_bytes(s, bare)});
    if (q.BM == 256 && q.KS == 1 && bare.KS == 1) break;
  }
  return std::max(most, align256((size_t)shape.T * shape.rank * 4));
}

hipError_t launch_adapter_linear(const moe_adapter_shape& s, const void* x, const void* W,
                                 const float* sc, const float* bias, const void* A, const void* B,
                                 const int32_t* ranks, const float* scales, const int32_t* idx,
                                 const void* base, void* y, void* ws, hipStream_t st) {
  const Plan q = plan_of(s, W != nullptr);
  AdapterParams p{};
  p.x = (const uint16_t*)x; p.W = W; p.s = sc; p.bias = bias;
  p.A = (const uint16_t*)A; p.B = (const uint16_t*)B; p.ranks = ranks; p.scales = scales;
  p.idx = idx; p.base = base; p.y = y; p.S = (float*)ws;
  p.part = (float*)((char*)ws + s_bytes(s, q));
  p.T = s.T; p.d_in = s.d_in; p.d_out = s.d_out; p.n = s.n_adapters; p.R = s.rank;
  p.y_f32 = s.y_dtype == MOE_DT_F32 ? 1 : 0;
  p.KS = q.KS; p.Z = q.Z; p.KW = q.KW;
  p.s_ranks = q.s_ranks; p.s_blocks = q.s_blocks;
  if (!W || q.BM == 256) {
    adapter_shrink_kernel<<<q.s_blocks, kThreads, 0, st>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (W) {
    const hipError_t e = launch_weights(s, p, q, st);
    if (e != hipSuccess || q.BM == 256) return e;
  }
  if (q.expand)
    adapter_expand_kernel<<<dim3((unsigned)((s.d_out + 127) / 128), (unsigned)((s.T + 31) / 32)),
                            kExpandThreads, 0, st>>>(p);
  else
    adapter_join_kernel<<<dim3((unsigned)((s.d_out + kJoin - 1) / kJoin), (unsigned)s.T), kJoin, 0,
                          st>>>(p);
  return hipGetLastError();
}

}  // namespace moe
