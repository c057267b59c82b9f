// Matrix product of 8-bit codes with a scale per token and per output channel, on INT8 MFMA.
//
// Both operands have their inner axis contiguous, as the matrix instructions take them (a lane's 16 codes are
// neighbours).  The weights are the instruction's first operand, so that a lane of the result holds 4 neighbouring output
// channels of one token and stores them together.
//
// Three kernels: few tokens are bound by the weights' bytes and streamed (1 x 4096 x 18560 15 us, 5.0 TB/s); many tokens
// by the matrix units and LDS together, which the tiles need for equally many cycles, at a clock that power limits (32768
// x 4096 x 18560 2.05 ms, 2.4 POP/s: matrix units at work in 58% of the cycles, at 1.9 GHz; out of registers alone random
// codes reach 3.4 to 4.0, zeros 4.8); inner sizes that no 16 divides by their unaligned loads (777 x 1531 x 1000 14 us).
#include <algorithm>

#include "block_internal.h"
#include "gated_types.h"

namespace ssdq {
namespace {

struct Epilogue {
  const float* a_scale;
  const float* b_scale;
  const float* bias;
  bool per_row;
};

// (float(sum) * a_scale) * b_scale + bias
__device__ __forceinline__ float finish(int32_t sum, float sa, float sb, float bias) {
  return fmaf(float(sum) * sa, sb, bias);
}

// 16 codes of a row of k, at any byte; those past the row's end are 0 and not read.
__device__ __forceinline__ v4i load_codes(const int8_t* __restrict__ row, int32_t at, int32_t k) {
  v4i r = {0, 0, 0, 0};
  if (at + 16 <= k) {
    __builtin_memcpy(&r, row + at, 16);
  } else if (at < k) {
    int8_t e[16] = {};
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (at + i < k) e[i] = row[at + i];
    __builtin_memcpy(&r, e, 16);
  }
  return r;
}

// Few tokens: the time is the weights' bytes.  A wave reads its part of 16 weight rows straight into the matrix
// instructions' operands, a whole 128-byte line of a row at a time, without LDS: four lanes per row take 32 bytes each, and
// the two halves of them enter two instructions (the sum does not mind which codes meet in which instruction, as long as
// both operands agree).  The waves of a block share the lines of the inner axis, and their sums meet in LDS.  Up to 16 MT
// tokens.  kAny: rows may start at any byte (1 x 8190 x 4096 19 us; by tiles 63).
constexpr int kLine = 128, kLinesAhead = 4;
constexpr int kStreamWaves = 16;              // at most

__device__ __forceinline__ v4i load_piece(Rsrc r, uint32_t offset) { return __builtin_bit_cast(v4i, buf_load16(r, offset)); }

template <typename T, int MT, bool kAny>
__global__ void __launch_bounds__(kStreamWaves* kWave)
    stream_kernel(const int8_t* __restrict__ a, const int8_t* __restrict__ b, Epilogue ep, T* __restrict__ out, int32_t m,
                  int32_t k, int32_t n) {
  extern __shared__ v4i sums[];   // [waves][MT][64]
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, waves = blockDim.x / kWave;
  const int32_t n0 = int32_t(blockIdx.x) * 16;
  const Rsrc ra = make_rsrc(a, uint32_t(m) * uint32_t(k));
  const Rsrc rb = make_rsrc(b + int64_t(n0) * k, uint32_t(min(n - n0, 16)) * uint32_t(k));
  const int32_t lines = (k + kLine - 1) / kLine;
  v4i acc[MT] = {};
  uint32_t row_at[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) row_at[i] = uint32_t(lane % 16 + 16 * i) * uint32_t(k);
  // Blocks begin at different lines: rows of many codes are often a power of two apart, and the same line of all rows
  // would lie in few of the memory's channels (1 x 4096 x 18560: 22 us, and 16 so).
  const int32_t turn = int32_t(blockIdx.x * 5 % uint32_t(lines));
  for (int32_t line0 = wave; line0 < lines; line0 += waves * kLinesAhead) {
    v4i fa[kLinesAhead][MT][2], fb[kLinesAhead][2];
#pragma unroll
    for (int l = 0; l < kLinesAhead; ++l) {
      int32_t line = line0 + l * waves;
      const bool some = line < lines;
      line += turn;
      if (line >= lines) line -= lines;
      const uint32_t at = some ? uint32_t(line) * kLine + (lane / 16) * 32 : kOutOfRange;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool in = at + h * 16 < uint32_t(k);
        if constexpr (kAny) {   // (rows past the last one: the last one's again, into results that are not stored)
          const int32_t from = in ? int32_t(at) + h * 16 : k;
          fb[l][h] = load_codes(b + int64_t(min(n0 + lane % 16, n - 1)) * k, from, k);
#pragma unroll
          for (int i = 0; i < MT; ++i) fa[l][i][h] = load_codes(a + int64_t(min(16 * i + lane % 16, m - 1)) * k, from, k);
        } else {
          fb[l][h] = load_piece(rb, in ? row_at[0] + at + h * 16 : kOutOfRange);
#pragma unroll
          for (int i = 0; i < MT; ++i) fa[l][i][h] = load_piece(ra, in ? row_at[i] + at + h * 16 : kOutOfRange);
        }
      }
    }
#pragma unroll
    for (int l = 0; l < kLinesAhead; ++l)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[l][h], fa[l][i][h], acc[i], 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) sums[(wave * MT + i) * kWave + lane] = acc[i];
  __syncthreads();
  if (wave >= MT) return;   // one wave for each 16 tokens
  v4i sum = {0, 0, 0, 0};
  for (int w = 0; w < waves; ++w) sum += sums[(w * MT + wave) * kWave + lane];
  const int32_t row = wave * 16 + lane % 16, col = n0 + (lane / 16) * 4;
  if (row >= m) return;
  const float sa = ep.a_scale[ep.per_row ? row : 0];
  T* to = out + int64_t(row) * n + col;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (col + e < n)
      to[e] = from_f32<T>(finish(sum[e], sa, ep.b_scale[col + e], ep.bias != nullptr ? ep.bias[col + e] : 0.f));
}

template <typename T, int MT, bool kAny = false>
hipError_t launch_stream(const MatmulArgs& a, const Epilogue& ep, hipStream_t stream) {
  const uint32_t blocks = uint32_t((int64_t(a.n) + 15) / 16);
  const int32_t lines = (a.k + kLine - 1) / kLine;
  int32_t waves = 4;
  while (waves < kStreamWaves && waves * kLinesAhead < lines && blocks * waves < 4096) waves *= 2;
  const size_t lds = size_t(waves) * MT * kWave * sizeof(v4i);
  stream_kernel<T, MT, kAny><<<dim3(blocks), waves * kWave, lds, stream>>>(a.a, a.b, ep, static_cast<T*>(a.out),
                                                                          int32_t(a.m), a.k, a.n);
  return hipGetLastError();
}

// Many tokens: tiles of TM tokens x TN output channels for inner sizes of whole 16-byte pieces.  Slabs of 128 codes of both
// operands, a whole line of every row, go from memory to LDS without passing registers and ahead of the products, into
// the next tile too: a block walks several tiles, and its loads do not stop between them (32768 x 4096 x 18560: through
// registers 4771 us, into LDS 3126, with the loads running on 2565, with the reads of LDS below 2046).
constexpr int kSlab = 128;

__device__ __forceinline__ void load_to_lds(Rsrc r, void* lds, uint32_t offset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, int(offset), 0, 0, 0);
}

// all but the newest N operations in memory have been done, and every read of LDS
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N < 64, "the counter has six bits");
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void barrier() {
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

struct TileArgs {
  const int8_t* a;
  const int8_t* b;
  Epilogue ep;
  int64_t m;
  int32_t k, n;
  uint32_t m_tiles, n_tiles;
};

// Consecutive blocks go to the 8 XCDs in turn.  An XCD takes a run of neighbouring tiles, walked in groups of 8 token
// tiles, so that the blocks that run together share rows in its L2; its blocks take the tiles of the run in turn.
template <int TM, int TN>
struct Walk {
  uint32_t run, before, stride, m_tiles, n_tiles;
  __device__ __forceinline__ Walk(const TileArgs& a) : m_tiles(a.m_tiles), n_tiles(a.n_tiles) {
    const uint32_t tiles = m_tiles * n_tiles, xcd = blockIdx.x % 8;
    run = tiles / 8 + (xcd < tiles % 8);
    before = xcd * (tiles / 8) + min(xcd, tiles % 8);
    stride = (gridDim.x + 7) / 8;
  }
  __device__ __forceinline__ void place(uint32_t t, int64_t& m0, int32_t& n0) const {
    constexpr uint32_t kGroup = 8;
    const uint32_t tile = before + t, group = tile / (kGroup * n_tiles), first = group * kGroup;
    const uint32_t height = min(m_tiles - first, kGroup), in_group = tile - first * n_tiles;
    m0 = int64_t(first + in_group % height) * TM;
    n0 = int32_t(in_group / height) * TN;
  }
};

// What a wave loads: 1 KB of rows of a slab at a time, 16 bytes a lane.  The pieces of a row are exchanged by the row's
// number, so that those which eight neighbouring rows give a matrix instruction lie in eight different places of 16 bytes.
__device__ __forceinline__ int place_of_piece(int row, int piece) { return piece ^ (row % 8); }

template <int TM, int TN, int kWaves>
struct Loader {
  static constexpr int kPieces = kSlab / 16, kRows = kWave / kPieces;   // pieces of a row, rows of a load
  static constexpr int LA = TM / kRows / kWaves, LB = TN / kRows / kWaves, kLoads = LA + LB;
  const TileArgs& a;
  const Walk<TM, TN>& walk;
  int wave;
  uint32_t tile, piece, row_at;
  int32_t slab, low, high, first, left, slabs;   // slabs [low, high) of a tile, from `first` on and round
  Rsrc ra, rb;
  // part `group` of `groups` equal ones of the slabs (the last may end in slabs past k, which load as zero)
  __device__ __forceinline__ Loader(const TileArgs& a, const Walk<TM, TN>& walk, int lane, int wave, int group, int groups)
      : a(a), walk(walk), wave(wave), tile(blockIdx.x / 8), piece(place_of_piece(lane / kPieces, lane % kPieces) * 16),
        row_at((uint32_t(wave) * kRows + lane / kPieces) * uint32_t(a.k)),
        slabs(((a.k + kSlab - 1) / kSlab + groups - 1) / groups) {
    low = group * slabs;
    high = low + slabs;
    // XCDs begin at different slabs: rows of many codes are often a power of two apart, and the same line of all rows
    // would lie in few of the memory's channels.
    first = low + int32_t(blockIdx.x % 8) * slabs / 8;
    aim();
  }
  __device__ __forceinline__ void aim() {
    slab = first;
    left = slabs;
    int64_t m0 = 0;
    int32_t n0 = 0;
    const bool some = tile < walk.run;   // past the last tile: nothing, zeros that nobody reads
    if (some) walk.place(tile, m0, n0);
    const int32_t rows_a = some ? int32_t(min(a.m - m0, int64_t(TM))) : 0, rows_b = some ? min(a.n - n0, TN) : 0;
    ra = make_rsrc(a.a + m0 * a.k, uint32_t(rows_a) * uint32_t(a.k));
    rb = make_rsrc(a.b + int64_t(n0) * a.k, uint32_t(rows_b) * uint32_t(a.k));
  }
  // the next slab into a stage of TM + TN rows
  __device__ __forceinline__ void operator()(int8_t* stage) {
    int8_t* to = stage + wave * 1024;
    const uint32_t at = uint32_t(slab) * kSlab + piece;
    const uint32_t from = at < uint32_t(a.k) ? row_at + at : kOutOfRange, step = uint32_t(kWaves * kRows) * uint32_t(a.k);
#pragma unroll
    for (int i = 0; i < LA; ++i) load_to_lds(ra, to + i * kWaves * 1024, from + i * step);
#pragma unroll
    for (int i = 0; i < LB; ++i) load_to_lds(rb, to + TM * kSlab + i * kWaves * 1024, from + i * step);
    if (++slab == high) slab = low;
    if (--left == 0) {
      tile += walk.stride;
      aim();
    }
  }
};

// A wave's share of a slab: FM x FN matrix instructions of 16 x 16, twice 64 codes.  All reads and their wait are one
// assembly statement: to reads of its own the compiler adds a wait for every load into LDS that is under way.
#define SSDQ_READ(to, from, row) "ds_read_b128 %" #to ", %" #from " offset:" #row "*2048\n\t"
template <int FM, int FN>
struct Operands {
  v4i a[2][FM], b[2][FN];
  // rows_a, rows_b: the wave's first rows of both operands
  __device__ __forceinline__ void read(const int8_t* rows_a, const int8_t* rows_b, int lane) {
    const uint32_t row = lane % 16, at0 = row * kSlab + place_of_piece(row, lane / 16) * 16, at1 = at0 ^ 64;
    typedef __attribute__((address_space(3))) const int8_t* Lds;
    const uint32_t pa = uint32_t(uintptr_t((Lds)rows_a)), pb = uint32_t(uintptr_t((Lds)rows_b));
    const uint32_t a0 = pa + at0, a1 = pa + at1, b0 = pb + at0, b1 = pb + at1;
    if constexpr (FM == 8 && FN == 4) {
      asm volatile(SSDQ_READ(16, 26, 0) SSDQ_READ(17, 26, 1) SSDQ_READ(18, 26, 2) SSDQ_READ(19, 26, 3)
                   SSDQ_READ(0, 24, 0) SSDQ_READ(1, 24, 1) SSDQ_READ(2, 24, 2) SSDQ_READ(3, 24, 3)
                   SSDQ_READ(4, 24, 4) SSDQ_READ(5, 24, 5) SSDQ_READ(6, 24, 6) SSDQ_READ(7, 24, 7)
                   SSDQ_READ(20, 27, 0) SSDQ_READ(21, 27, 1) SSDQ_READ(22, 27, 2) SSDQ_READ(23, 27, 3)
                   SSDQ_READ(8, 25, 0) SSDQ_READ(9, 25, 1) SSDQ_READ(10, 25, 2) SSDQ_READ(11, 25, 3)
                   SSDQ_READ(12, 25, 4) SSDQ_READ(13, 25, 5) SSDQ_READ(14, 25, 6) SSDQ_READ(15, 25, 7)
                   "s_waitcnt lgkmcnt(0)"
                   : "=&v"(a[0][0]), "=&v"(a[0][1]), "=&v"(a[0][2]), "=&v"(a[0][3]), "=&v"(a[0][4]), "=&v"(a[0][5]),
                     "=&v"(a[0][6]), "=&v"(a[0][7]), "=&v"(a[1][0]), "=&v"(a[1][1]), "=&v"(a[1][2]), "=&v"(a[1][3]),
                     "=&v"(a[1][4]), "=&v"(a[1][5]), "=&v"(a[1][6]), "=&v"(a[1][7]), "=&v"(b[0][0]), "=&v"(b[0][1]),
                     "=&v"(b[0][2]), "=&v"(b[0][3]), "=&v"(b[1][0]), "=&v"(b[1][1]), "=&v"(b[1][2]), "=&v"(b[1][3])
                   : "v"(a0), "v"(a1), "v"(b0), "v"(b1)
                   : "memory");
    } else if constexpr (FM == 4 && FN == 4) {
      asm volatile(SSDQ_READ(8, 18, 0) SSDQ_READ(9, 18, 1) SSDQ_READ(10, 18, 2) SSDQ_READ(11, 18, 3)
                   SSDQ_READ(0, 16, 0) SSDQ_READ(1, 16, 1) SSDQ_READ(2, 16, 2) SSDQ_READ(3, 16, 3)
                   SSDQ_READ(12, 19, 0) SSDQ_READ(13, 19, 1) SSDQ_READ(14, 19, 2) SSDQ_READ(15, 19, 3)
                   SSDQ_READ(4, 17, 0) SSDQ_READ(5, 17, 1) SSDQ_READ(6, 17, 2) SSDQ_READ(7, 17, 3)
                   "s_waitcnt lgkmcnt(0)"
                   : "=&v"(a[0][0]), "=&v"(a[0][1]), "=&v"(a[0][2]), "=&v"(a[0][3]), "=&v"(a[1][0]), "=&v"(a[1][1]),
                     "=&v"(a[1][2]), "=&v"(a[1][3]), "=&v"(b[0][0]), "=&v"(b[0][1]), "=&v"(b[0][2]), "=&v"(b[0][3]),
                     "=&v"(b[1][0]), "=&v"(b[1][1]), "=&v"(b[1][2]), "=&v"(b[1][3])
                   : "v"(a0), "v"(a1), "v"(b0), "v"(b1)
                   : "memory");
    } else if constexpr (FM == 4 && FN == 2) {
      asm volatile(SSDQ_READ(8, 14, 0) SSDQ_READ(9, 14, 1)
                   SSDQ_READ(0, 12, 0) SSDQ_READ(1, 12, 1) SSDQ_READ(2, 12, 2) SSDQ_READ(3, 12, 3)
                   SSDQ_READ(10, 15, 0) SSDQ_READ(11, 15, 1)
                   SSDQ_READ(4, 13, 0) SSDQ_READ(5, 13, 1) SSDQ_READ(6, 13, 2) SSDQ_READ(7, 13, 3)
                   "s_waitcnt lgkmcnt(0)"
                   : "=&v"(a[0][0]), "=&v"(a[0][1]), "=&v"(a[0][2]), "=&v"(a[0][3]), "=&v"(a[1][0]), "=&v"(a[1][1]),
                     "=&v"(a[1][2]), "=&v"(a[1][3]), "=&v"(b[0][0]), "=&v"(b[0][1]), "=&v"(b[1][0]), "=&v"(b[1][1])
                   : "v"(a0), "v"(a1), "v"(b0), "v"(b1)
                   : "memory");
    } else {
      static_assert(FM == 2 && FN == 2, "a wave's tiles");
      asm volatile(SSDQ_READ(4, 10, 0) SSDQ_READ(5, 10, 1) SSDQ_READ(0, 8, 0) SSDQ_READ(1, 8, 1)
                   SSDQ_READ(6, 11, 0) SSDQ_READ(7, 11, 1) SSDQ_READ(2, 9, 0) SSDQ_READ(3, 9, 1)
                   "s_waitcnt lgkmcnt(0)"
                   : "=&v"(a[0][0]), "=&v"(a[0][1]), "=&v"(a[1][0]), "=&v"(a[1][1]), "=&v"(b[0][0]), "=&v"(b[0][1]),
                     "=&v"(b[1][0]), "=&v"(b[1][1])
                   : "v"(a0), "v"(a1), "v"(b0), "v"(b1)
                   : "memory");
    }
  }
  __device__ __forceinline__ void multiply(v4i (&acc)[FN][FM]) const {
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          acc[j][i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[half][j], a[half][i], acc[j][i], 0, 0, 0);
  }
};
#undef SSDQ_READ

// A wave's results, 16 FM tokens x 16 FN channels from (row0, col0) on, to memory.  They pass through LDS, 16 tokens x 128
// bytes at a time, to be stored in whole lines.  Returns whether all of it was stored, in kStores instructions.
template <typename T, int FM, int FN>
struct Store {
  static constexpr int kUnit = FN * 16 * int(sizeof(T)) < 128 ? FN * 16 : 128 / int(sizeof(T));   // channels at a time
  static constexpr int kUnits = FN * 16 / kUnit, kBytes = kUnit * int(sizeof(T)), kPitch = kBytes + 16;
  static constexpr int kLanes = kBytes / 16, kRows = kWave / kLanes, kParts = 16 / kRows;   // of a store instruction
  static constexpr int kStores = FM * kUnits * kParts, kRoom = 16 * kPitch;
  static_assert(kParts >= 1 && kUnit % 16 == 0, "a store instruction takes whole rows");
  __device__ __forceinline__ static bool run(const v4i (&acc)[FN][FM], const TileArgs& a, T* __restrict__ out,
                                             int8_t* room, int lane, int64_t row0, int32_t col0) {
    // a lane holds 4 neighbouring channels, col + 16 j, of the tokens row + 16 i
    float sb[FN][4], bias[FN][4], sa[FM];
    const int32_t col = col0 + (lane / 16) * 4;
    const int64_t row = row0 + lane % 16;
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int32_t c = min(col + j * 16 + e, a.n - 1);
        sb[j][e] = a.ep.b_scale[c];
        bias[j][e] = a.ep.bias != nullptr ? a.ep.bias[c] : 0.f;
      }
#pragma unroll
    for (int i = 0; i < FM; ++i) sa[i] = a.ep.a_scale[a.ep.per_row ? min(row + i * 16, a.m - 1) : 0];
    struct Four { T e[4]; };
    const bool whole = row0 + FM * 16 <= a.m && col0 + FN * 16 <= a.n;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
#pragma unroll
      for (int part = 0; part < kUnits; ++part) {
#pragma unroll
        for (int j = 0; j < FN / kUnits; ++j) {
          const int jj = part * (FN / kUnits) + j;
          Four r;
#pragma unroll
          for (int e = 0; e < 4; ++e) r.e[e] = from_f32<T>(finish(acc[jj][i][e], sa[i], sb[jj][e], bias[jj][e]));
          *reinterpret_cast<Four*>(room + (lane % 16) * kPitch + (j * 16 + (lane / 16) * 4) * sizeof(T)) = r;
        }
        // (a wave's reads of LDS follow its writes in order)
#pragma unroll
        for (int h = 0; h < kParts; ++h) {
          const int r = h * kRows + lane / kLanes;
          const v4i line = *reinterpret_cast<const v4i*>(room + r * kPitch + (lane % kLanes) * 16);
          const int64_t to_row = row0 + i * 16 + r;
          const int32_t to_col = col0 + part * kUnit + (lane % kLanes) * (16 / int(sizeof(T)));
          T* to = out + to_row * a.n + to_col;
          if (whole) {
            __builtin_memcpy(to, &line, 16);
          } else if (to_row < a.m) {
            struct { T e[16 / sizeof(T)]; } some;
            __builtin_memcpy(&some, &line, 16);
#pragma unroll
            for (int e = 0; e < int(16 / sizeof(T)); ++e)
              if (to_col + e < a.n) to[e] = some.e[e];
          }
        }
      }
    }
    return whole;
  }
};

// WM x WN waves, kStages slabs in LDS.  Between two barriers every wave reads a slab's operands and multiplies them.  The
// largest tiles read the fewest bytes of LDS per product: a slab of 256 x 256 in 8 waves takes the matrix units and LDS
// (reads and arriving loads) 2048 cycles each; 64 x 64 is bound by LDS and by what a compute unit can load (256 x 8192 x
// 4096 16.5 to 20 us, 1 POP/s).  With
// kSplit 2 there are twice the waves, and the halves of them walk half of the inner axis each: two waves on every SIMD for
// tiles that are too few to give a compute unit a second one.
template <typename T, int TM, int TN, int WM, int WN, int kStages, int kSplit>
__global__ void __launch_bounds__(WM * WN * kSplit * kWave) tile_kernel(TileArgs args, T* __restrict__ out) {
  constexpr int kWaves = WM * WN, FM = TM / WM / 16, FN = TN / WN / 16;
  typedef Loader<TM, TN, kWaves> Load;
  typedef Store<T, FM, FN> Put;
  constexpr int kAhead = (kStages - 2) * Load::kLoads;
  constexpr int kAheadStored = kAhead + Put::kStores < 63 ? kAhead + Put::kStores : 63;
  __shared__ __attribute__((aligned(16))) int8_t lds[kSplit][kStages][(TM + TN) * kSlab];
  __shared__ __attribute__((aligned(16))) int8_t results[kWaves][Put::kRoom];
  __shared__ v4i sums[kSplit > 1 ? kWaves : 1][kSplit > 1 ? FM * FN : 1][kWave];
  const int lane = threadIdx.x % kWave, of_block = __builtin_amdgcn_readfirstlane(int(threadIdx.x / kWave));
  const int group = of_block / kWaves, wave = of_block % kWaves;
  const Walk<TM, TN> walk(args);
  Load load(args, walk, lane, wave, group, kSplit);
  const int wm = (wave % WM) * (TM / WM), wn = (wave / WM) * (TN / WN);
#pragma unroll
  for (int i = 0; i + 1 < kStages; ++i) load(lds[group][i]);
  int stage = 0;
  bool stored = false;   // whether the newest operations in memory are the stores of a whole tile
  for (uint32_t t = blockIdx.x / 8; t < walk.run; t += walk.stride) {
    v4i acc[FN][FM] = {};
    for (int32_t slab = 0; slab < load.slabs; ++slab) {
      // This wave's part of the slab has arrived; behind the barrier all parts have, and the slab before has been read
      // by all waves: its stage takes the newest loads.  (Loads and stores count in order: the loads of a tile's first
      // slabs were issued ahead of the stores of the tile before.)
      if (stored && slab < kStages - 1) wait_loads<kAheadStored>();
      else wait_loads<kAhead>();
      barrier();
      load(lds[group][stage == 0 ? kStages - 1 : stage - 1]);
      Operands<FM, FN> o;
      o.read(lds[group][stage] + wm * kSlab, lds[group][stage] + (TM + wn) * kSlab, lane);
      o.multiply(acc);
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    if constexpr (kSplit > 1) {
      if (group == 1) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int i = 0; i < FM; ++i) sums[wave][j * FM + i][lane] = acc[j][i];
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      barrier();
      if (group == 1) continue;
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int i = 0; i < FM; ++i) acc[j][i] += sums[wave][j * FM + i][lane];
    }
    int64_t m0;
    int32_t n0;
    walk.place(t, m0, n0);
    stored = Put::run(acc, args, out, results[wave], lane, m0 + wm, n0 + wn);
  }
  wait_loads<0>();   // no load is under way into LDS that another block may have
}

// Inner sizes of any number of codes: rows may start at any byte, so the pieces pass through registers, those of the next
// slabs while the current one is multiplied (loads of 16 bytes at any address, which take five times as long as aligned
// ones and bound the kernel; the aligned words that hold them, shifted, take longer still: 777 x 1531 x 1000 18.2 us
// against 15.3).  A row's last slab is loaded code by code.  Square tiles, 4 waves, of 128 once there is one for every
// compute unit (8192 x 4097 x 8192 501 us, 862 with 64), else of 64; those no more than compute units in two halves of
// the inner axis as above (777 x 1531 x 1000 14.8 and 13.8 us so, 64 x 8190 x 4096 46.5 and 37.2, 300 x 100 x 700 9.7 and
// 9.8).
template <typename T, int kSide, int kSplit>
__global__ void __launch_bounds__(256 * kSplit) ragged_kernel(TileArgs args, T* __restrict__ out) {
  constexpr int kThreads = 256, kPieces = 2 * kSide * kSlab / 16 / kThreads, F = kSide / 32;
  constexpr int kSets = kSide == 64 ? 2 : 1;   // slabs in registers
  typedef Store<T, F, F> Put;
  __shared__ __attribute__((aligned(16))) int8_t lds[kSplit][2][2 * kSide * kSlab];
  __shared__ __attribute__((aligned(16))) int8_t results[4][Put::kRoom];
  __shared__ v4i sums[kSplit > 1 ? 4 : 1][kSplit > 1 ? F * F : 1][kWave];
  const int lane = threadIdx.x % kWave, of_block = __builtin_amdgcn_readfirstlane(int(threadIdx.x / kWave));
  const int group = of_block / 4, wave = of_block % 4, thread = threadIdx.x % kThreads;
  const Walk<kSide, kSide> walk(args);
  const int wm = (wave % 2) * (kSide / 2), wn = (wave / 2) * (kSide / 2), piece = thread % 8;
  const int32_t slabs = ((args.k + kSlab - 1) / kSlab + kSplit - 1) / kSplit;   // (the last may be past k: zeros)
  for (uint32_t t = blockIdx.x / 8; t < walk.run; t += walk.stride) {
    int64_t m0;
    int32_t n0;
    walk.place(t, m0, n0);
    const int8_t* row[kPieces];
    v4i pieces[kSets][kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int r = thread / 8 + i * (kThreads / 8);   // the tokens' rows, then the channels'
      row[i] = r < kSide ? args.a + min(m0 + r, args.m - 1) * args.k
                         : args.b + int64_t(min(n0 + r - kSide, args.n - 1)) * args.k;
    }
    const auto load = [&](int32_t of_group, int set) __attribute__((always_inline)) {
      const int32_t slab = group * slabs + of_group;
      if ((slab + 1) * kSlab <= args.k) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) __builtin_memcpy(&pieces[set][i], row[i] + slab * kSlab + piece * 16, 16);
      } else {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) pieces[set][i] = load_codes(row[i], slab * kSlab + piece * 16, args.k);
      }
    };
    v4i acc[F][F] = {};
    const auto multiply = [&](int32_t slab, int set) __attribute__((always_inline)) {
      int8_t* rows = lds[group][slab & 1];
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int r = thread / 8 + i * (kThreads / 8);
        *reinterpret_cast<v4i*>(rows + r * kSlab + place_of_piece(r, piece) * 16) = pieces[set][i];
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      barrier();
      if (slab + kSets < slabs) load(slab + kSets, set);
      Operands<F, F> o;
      o.read(rows + wm * kSlab, rows + (kSide + wn) * kSlab, lane);
      o.multiply(acc);
    };
#pragma unroll
    for (int i = 0; i < kSets; ++i)
      if (i < slabs) load(i, i);
    for (int32_t slab = 0; slab < slabs; slab += kSets) {
      multiply(slab, 0);
      if (kSets > 1 && slab + 1 < slabs) multiply(slab + 1, kSets - 1);
    }
    if constexpr (kSplit > 1) {
      if (group == 1) {
#pragma unroll
        for (int j = 0; j < F; ++j)
#pragma unroll
          for (int i = 0; i < F; ++i) sums[wave][j * F + i][lane] = acc[j][i];
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      barrier();
      if (group == 0) {
#pragma unroll
        for (int j = 0; j < F; ++j)
#pragma unroll
          for (int i = 0; i < F; ++i) acc[j][i] += sums[wave][j * F + i][lane];
      }
    }
    if (group == 0) Put::run(acc, args, out, results[wave], lane, m0 + wm, n0 + wn);
    barrier();   // the next tile's first slab goes over one that other waves may still read
  }
}

template <int TM, int TN>
TileArgs tile_args(const MatmulArgs& a, const Epilogue& ep, int per_unit, uint32_t* blocks) {
  const uint32_t m_tiles = uint32_t((a.m + TM - 1) / TM), n_tiles = uint32_t((int64_t(a.n) + TN - 1) / TN);
  const int32_t units = std::max(8, compute_units() / 8 * 8);   // the same number on every XCD
  *blocks = std::min(m_tiles * n_tiles, uint32_t(units * per_unit));
  return TileArgs{a.a, a.b, ep, a.m, a.k, a.n, m_tiles, n_tiles};
}

// `per_unit` blocks on a compute unit
template <typename T, int TM, int TN, int WM, int WN, int kStages, int kSplit = 1>
hipError_t launch_tiles(const MatmulArgs& a, const Epilogue& ep, int per_unit, hipStream_t stream) {
  uint32_t blocks;
  const TileArgs args = tile_args<TM, TN>(a, ep, per_unit, &blocks);
  tile_kernel<T, TM, TN, WM, WN, kStages, kSplit>
      <<<dim3(blocks), WM * WN * kSplit * kWave, 0, stream>>>(args, static_cast<T*>(a.out));
  return hipGetLastError();
}

// Which tiles: the fewest microseconds by rounds x slabs x the time of a slab, where a round is as many tiles as the device
// holds at once with 16-bit output and the times are those measured with all compute units at work.  (With fp32 output a
// block of 128 x 64 tiles has 82944 bytes of LDS, of which a compute unit holds one and not two; its rounds count as if it
// held two: 1024 x 4096 x 4096 34 to 37 us, with fp16 output 23.5; 128 x 4096 x 18560 32 to 33 and 21.8.)
struct Candidate { int32_t plan; int tm, tn, per_unit; float slab_us; };
constexpr Candidate kCandidates[] = {{SSDQ_MATMUL_TILES_256X256, 256, 256, 1, 1.80f}, {SSDQ_MATMUL_TILES_128X128, 128, 128, 2, 1.06f},
                                     {SSDQ_MATMUL_TILES_128X64, 128, 64, 2, 0.68f}, {SSDQ_MATMUL_TILES_64X64, 64, 64, 2, 0.50f}};

int32_t choose(int64_t m, int32_t n) {
  int best = 0;
  double least = 0.;
  for (int i = 0; i < 4; ++i) {
    const Candidate& c = kCandidates[i];
    const int64_t tiles = (m + c.tm - 1) / c.tm * ((int64_t(n) + c.tn - 1) / c.tn);
    const int64_t slots = int64_t(compute_units()) * c.per_unit;
    const double time = double((tiles + slots - 1) / slots) * c.slab_us;
    if (i == 0 || time < least) {
      best = i;
      least = time;
    }
  }
  return kCandidates[best].plan;
}

template <typename T, int kSide, int kSplit>
hipError_t launch_ragged(const MatmulArgs& a, const Epilogue& ep, int per_unit, hipStream_t stream) {
  uint32_t blocks;
  const TileArgs args = tile_args<kSide, kSide>(a, ep, per_unit, &blocks);
  ragged_kernel<T, kSide, kSplit><<<dim3(blocks), 256 * kSplit, 0, stream>>>(args, static_cast<T*>(a.out));
  return hipGetLastError();
}

template <typename T>
hipError_t launch(const MatmulArgs& a, hipStream_t stream) {
  const Epilogue ep = {a.a_scale, a.b_scale, a.bias, a.per_row};
  switch (matmul_i8_plan(a.m, a.k, a.n)) {
    case SSDQ_MATMUL_STREAM_16: return launch_stream<T, 1>(a, ep, stream);
    case SSDQ_MATMUL_STREAM_32: return launch_stream<T, 2>(a, ep, stream);
    case SSDQ_MATMUL_TILES_256X256: return launch_tiles<T, 256, 256, 2, 4, 2>(a, ep, kCandidates[0].per_unit, stream);
    case SSDQ_MATMUL_TILES_128X128: return launch_tiles<T, 128, 128, 2, 2, 2>(a, ep, kCandidates[1].per_unit, stream);
    case SSDQ_MATMUL_TILES_128X64: return launch_tiles<T, 128, 64, 2, 2, 3>(a, ep, kCandidates[2].per_unit, stream);
    case SSDQ_MATMUL_TILES_64X64: return launch_tiles<T, 64, 64, 2, 2, 4>(a, ep, kCandidates[3].per_unit, stream);
    case SSDQ_MATMUL_TILES_64X64_HALVES: return launch_tiles<T, 64, 64, 2, 2, 4, 2>(a, ep, 1, stream);
    case SSDQ_MATMUL_ODD_STREAM_16: return launch_stream<T, 1, true>(a, ep, stream);
    case SSDQ_MATMUL_ODD_128X128: return launch_ragged<T, 128, 1>(a, ep, 2, stream);
    case SSDQ_MATMUL_ODD_64X64: return launch_ragged<T, 64, 1>(a, ep, 3, stream);
    default: return launch_ragged<T, 64, 2>(a, ep, 1, stream);
  }
}

}  // namespace

int32_t matmul_i8_plan(int64_t m, int32_t k, int32_t n) {
  const int64_t tiles = (m + 63) / 64 * ((int64_t(n) + 63) / 64);   // of the smallest size
  if (k % 16 != 0) {
    if (m <= 16 && n <= 1 << 24) return SSDQ_MATMUL_ODD_STREAM_16;
    if ((m + 127) / 128 * ((int64_t(n) + 127) / 128) >= compute_units()) return SSDQ_MATMUL_ODD_128X128;
    return tiles > compute_units() ? SSDQ_MATMUL_ODD_64X64 : SSDQ_MATMUL_ODD_64X64_HALVES;
  }
  // Few tokens: up to 8 the tokens' bytes are nothing beside the weights'; up to 32 where tiles of 64 channels would leave
  // half of the compute units idle (16 x 8192 x 4096: 11.0 us against 20.5; 16 x 4096 x 18560: 23.2 against 20.9).
  const bool narrow = (int64_t(n) + 63) / 64 * 2 <= compute_units();
  if ((m <= 8 && n <= 1 << 24) || (m <= 16 && narrow)) return SSDQ_MATMUL_STREAM_16;
  if (m <= 32 && narrow) return SSDQ_MATMUL_STREAM_32;
  const int32_t best = choose(m, n);
  // no more tiles than compute units: two halves of the inner axis in each (256 x 4096 x 4096 12.9 us and 11.2 so;
  // 64 x 4096 x 18560, 290 tiles, 24.0 and 24.5)
  return best == SSDQ_MATMUL_TILES_64X64 && tiles <= compute_units() ? SSDQ_MATMUL_TILES_64X64_HALVES : best;
}

hipError_t launch_matmul_i8(const MatmulArgs& a, hipStream_t stream) {
  switch (a.dtype) {
    case SSDQ_DTYPE_F32: return launch<float>(a, stream);
    case SSDQ_DTYPE_F16: return launch<_Float16>(a, stream);
    default: return launch<__bf16>(a, stream);
  }
}

}  // namespace ssdq
