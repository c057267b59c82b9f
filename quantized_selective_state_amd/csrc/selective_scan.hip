// Selective state space scan: a decay for every (channel, state) and a step size for every channel, for prompts (dense
// or packed) and for single tokens.
//
//   d = softplus(delta + bias);  h[n] = exp(d A[n]) h[n] + d u B[n];  y = (sum_n C[n] h[n] + D u) silu(z)
//
// Two ways to walk. Dense sequences whole, by four lanes a channel with a quarter of its states each (quad_kernel): one
// pass, where sequences and channels give the device enough waves or the sequences are short.  Otherwise, and packed, in
// chunks of rows side by side (chunk_kernel), a lane holding one channel with up to 16 states: a first kernel forms what
// every chunk makes of a zero state, a second one carries states from chunk to chunk, h <- exp(A sum d) h + that, and a
// third walks the chunks again from the states that enter them and writes y.  B and C, the same for all channels, are
// staged as binary32 in LDS.
//
// Bound by the vector units, not by memory: a token, channel and state costs an exp2 (a third of the rate of an fma), two
// products, an fma into the state and one into y.  With 16 states, bf16: 4 x 2048 x 4096 219 us (its bytes would take 54; in
// chunks 255), 16 x 2048 x 8192 1050 us (4.1e12 tokens x channels x states a second).  16384 x 5120 fp16, in chunks, 577 us.
// 4 x 2048 x 4096 with 64 states 535 us (in chunks 1255).
//
// exp(d A) is the hardware's exp2 of d (A log2(e)), two rounded products of a rounded constant, for all types: within
// (2.3 |d A| + 3) 2^-24 of itself (measured 2.1 (|d A| + 1)), where the pair of exp_f32<true> would be within 3.  That
// relative error is large only where the decay is small.  Errors that add up are those of decays near 1, whose |d A| is
// near 0: a state that lives for 1 / |d A| tokens collects some 2^-24 in each, as its own roundings do.
#include "block_internal.h"
#include "gated_types.h"
#include "sequences.h"

namespace ssdq {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 16;            // rows of B and C in LDS at a time
constexpr int kGroup = 4;            // rows whose values are loaded together, one group ahead
constexpr float kLog2e = 1.44269502e+00f;

// softplus(v) = max(v, 0) + log(1 + e), e = exp(-|v|).  With w the rounded 1 + e, log(1 + e) is log(w) and about what the
// rounding left, e - (w - 1): wrong by no more than 2^-24 of itself, so that also small step sizes keep their relative
// precision.  -inf gives 0.
template <bool EXACT>
__device__ __forceinline__ float softplus(float v) {
  const float e = exp_f32<EXACT>(-fabsf(v)), w = 1.f + e, left = e - (w - 1.f);
  return fmaf(__builtin_amdgcn_logf(w), 6.93147182e-01f, left) + fmaxf(v, 0.f);   // (a NaN stays one: e is one)
}

// One element of a lane at `lane` bytes, `row` bytes (the same for all lanes) into a buffer.
template <typename T>
__device__ __forceinline__ T load_element(Rsrc r, uint32_t lane, uint32_t row) {
  if constexpr (sizeof(T) == 4) return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b32(r, int(lane), int(row), 0));
  else return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b16(r, int(lane), int(row), 0));
}
template <typename T>
__device__ __forceinline__ void store_element(Rsrc r, uint32_t lane, uint32_t row, T v) {
  if constexpr (sizeof(T) == 4) __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), r, int(lane), int(row), 0);
  else __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(u16, v), r, int(lane), int(row), 0);
}

// N states from `first` on, `pitch` elements apart, all loaded before the first is looked at; those past dstate are 0.
template <int N>
__device__ __forceinline__ void load_states(const float* __restrict__ p, int64_t pitch, int first, int dstate, float (&v)[N]) {
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = p[min(first + n, dstate - 1) * pitch];
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = first + n < dstate ? v[n] : 0.f;
}

struct ScanKernelArgs {
  Sequences seq;
  const void* u;
  const void* delta;
  const float* A;
  const void* B;
  const void* C;
  const float* D;
  const void* z;
  const float* delta_bias;
  const float* h0;
  void* y;
  float* h_final;
  float* states;       // (chunks, N, channels): after the first kernel a chunk's own, after the second what leaves it
  float* sums;         // (chunks, channels): sum of d over the chunk
  int32_t* resets;     // (chunks): what leaves the chunk does not depend on what enters it
  int32_t channels, dstate;
  int32_t chunk;       // rows
  int32_t per_sequence;   // chunks of a dense sequence; packed: all
  int32_t chunks;
  bool softplus;
};

// the rows of a chunk: dense chunks are cut within their sequence, packed ones at multiples of the chunk
__device__ __forceinline__ Span chunk_rows(const ScanKernelArgs& a, int32_t k) {
  if (a.seq.offsets != nullptr) return Span{k * a.chunk, int32_t(min(int64_t(k + 1) * a.chunk, int64_t(a.seq.tokens)))};
  const int32_t s = k / a.per_sequence, i = k - s * a.per_sequence;
  const Span span = a.seq.span(s);
  return Span{span.begin + i * a.chunk, int32_t(min(int64_t(span.begin) + int64_t(i + 1) * a.chunk, int64_t(span.end)))};
}

// The first kernel (OUTPUT false) forms what leaves a chunk by itself, the third one y and the final states.
//
// Of a block's four waves G share 64 channels, with N of the states each; their parts of C . h meet in LDS.  The products
// d u B[n] and their sum with exp(d A) h come from the matrix unit: one 4 x 4 x 1 instruction of 16 blocks is, for the 64
// channels of the lanes, an outer product of 4 states of B and d u, added to 4 registers of each lane.  That takes an fma
// and the read of B in every lane off the vector units (a row of 64 channels x 16 states, in cycles of a wave on its own:
// 318 against 365 with fma, with y 398 against 445; the instruction's sums are binary32 like an fma's).  Vector units are
// at work in 84 and 86% of the cycles (16384 x 5120 fp16: 258 us without y, 347 with it).
template <typename T, int N, int G, bool OUTPUT>
__global__ void __launch_bounds__(kThreads, OUTPUT ? 3 : 4) chunk_kernel(ScanKernelArgs a) {
  constexpr bool EXACT = sizeof(T) == 4;
  constexpr int kChannels = kThreads / G, kStates = N * G;
  constexpr int kPer = (kRows * kStates + kThreads - 1) / kThreads;   // values of B, and of C, that a thread stages
  __shared__ __attribute__((aligned(16))) float Bs[2][kRows][G][4][N / 4];   // state 4 q + i of a wave at [i][q]
  __shared__ __attribute__((aligned(16))) float Cs[OUTPUT ? 2 : 1][OUTPUT ? kRows : 1][kStates];
  __shared__ float parts[OUTPUT && G > 1 ? kRows : 1][G][OUTPUT && G > 1 ? kChannels : 1];
  const int lane = int(threadIdx.x) % kWave, wave = int(threadIdx.x) / kWave;
  const int group = wave % G, first_state = group * N;
  const int32_t block_channel = int32_t(blockIdx.y) * kChannels, c = block_channel + wave / G * kWave + lane;
  const bool live = c < a.channels;
  const int32_t cc = min(c, a.channels - 1);   // lanes past the last channel compute it too and store nothing
  if (int32_t(blockIdx.x) >= a.chunks) {       // sequences without rows: their state passes through
    const int32_t step = int32_t(gridDim.x) - a.chunks;
    for (int32_t s = int32_t(blockIdx.x) - a.chunks; s < a.seq.sequences; s += step) {
      const Span span = a.seq.span(s);
      if (span.begin < span.end || !live) continue;
      for (int n = first_state; n < min(a.dstate, first_state + N); ++n) {
        const int64_t at = (int64_t(s) * a.channels + c) * a.dstate + n;
        a.h_final[at] = a.h0 != nullptr ? a.h0[at] : 0.f;
      }
    }
    return;
  }
  const int32_t k = int32_t(blockIdx.x);
  const Span rows = chunk_rows(a, k);
  // (without OUTPUT only what leaves the chunk is wanted: the sequence of its last row, where that goes on behind it)
  int32_t s = a.seq.at(OUTPUT ? rows.begin : rows.end - 1);
  Span span = a.seq.span(s);
  int32_t from = rows.begin;
  if constexpr (!OUTPUT) {
    const bool leaves = span.begin < rows.end && span.end > rows.end;
    if (blockIdx.y == 0 && threadIdx.x == 0) a.resets[k] = !leaves || span.begin >= rows.begin;
    if (!leaves) return;
    from = max(from, span.begin);
  }
  float A2[N], sum = 0.f;
  v4f h[N / 4] = {};
  load_states<N>(a.A + int64_t(cc) * a.dstate, 1, first_state, a.dstate, A2);
#pragma unroll
  for (int n = 0; n < N; ++n) A2[n] *= kLog2e;
  const float bias = a.delta_bias != nullptr ? a.delta_bias[cc] : 0.f;
  const float skip = OUTPUT && a.D != nullptr ? a.D[cc] : 0.f;
  // the chunk's rows of u, delta, z and y; lanes past the last channel store nowhere
  const int64_t base = int64_t(rows.begin) * a.channels;
  const uint32_t pitch = uint32_t(a.channels) * sizeof(T), bytes = uint32_t(rows.end - rows.begin) * pitch;
  const uint32_t at_lane = uint32_t(cc) * sizeof(T), store_lane = live ? at_lane : kOutOfRange;
  const bool has_z = OUTPUT && a.z != nullptr;
  const Rsrc ru = make_rsrc(static_cast<const T*>(a.u) + base, bytes), rd = make_rsrc(static_cast<const T*>(a.delta) + base, bytes);
  const Rsrc rz = make_rsrc(static_cast<const T*>(has_z ? a.z : a.u) + base, bytes);
  const Rsrc ry = make_rsrc(static_cast<T*>(a.y) + base, OUTPUT ? bytes : 0u);
  const uint32_t row_bytes = uint32_t(a.dstate) * sizeof(T), bc_bytes = uint32_t(rows.end - rows.begin) * row_bytes;
  const Rsrc rB = make_rsrc(static_cast<const T*>(a.B) + int64_t(rows.begin) * a.dstate, bc_bytes);
  const Rsrc rC = make_rsrc(static_cast<const T*>(a.C) + int64_t(rows.begin) * a.dstate, bc_bytes);

  const auto enter = [&](int32_t row) {   // the state ahead of `row`, which is in sequence s
    if (row != span.begin && !(OUTPUT && k > 0)) return;   // (k is 0 here only with offsets out of order)
    float v[N] = {};
    if (row != span.begin)
      load_states<N>(a.states + int64_t(k - 1) * a.dstate * a.channels + cc, a.channels, first_state, a.dstate, v);
    else if (a.h0 != nullptr)
      load_states<N>(a.h0 + (int64_t(s) * a.channels + cc) * a.dstate, 1, first_state, a.dstate, v);
#pragma unroll
    for (int n = 0; n < N; ++n) h[n / 4][n % 4] = v[n];
  };
  const auto leave = [&]() {
    if (!OUTPUT || !live || a.h_final == nullptr) return;
#pragma unroll
    for (int n = 0; n < N; ++n)
      if (first_state + n < a.dstate)
        a.h_final[(int64_t(s) * a.channels + c) * a.dstate + first_state + n] = h[n / 4][n % 4];
  };
  // a row of B and C as a token needs it
  struct Row { float b[N / 4]; v4f c[OUTPUT ? N / 4 : 1]; };
  const auto read_row = [&](int buffer, int r) __attribute__((always_inline)) {
    Row t;
    __builtin_memcpy(t.b, __builtin_assume_aligned(&Bs[buffer][r][group][lane % 4][0], N), N);
    if constexpr (OUTPUT) {
#pragma unroll
      for (int q = 0; q < N / 4; ++q) t.c[q] = *reinterpret_cast<const v4f*>(&Cs[buffer][r][first_state + 4 * q]);
    }
    return t;
  };
  // one token: d its step size, v its u; returns C . h
  const auto token = [&](float d, float v, const Row& t) __attribute__((always_inline)) {
    const float dv = d * v;
    float out[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int q = 0; q < N / 4; ++q) {
#pragma unroll
      for (int i = 0; i < 4; ++i) h[q][i] *= __builtin_amdgcn_exp2f(d * A2[4 * q + i]);
      h[q] = __builtin_amdgcn_mfma_f32_4x4x1f32(t.b[q], dv, h[q], 0, 0, 0);
    }
    if constexpr (OUTPUT) {
#pragma unroll
      for (int q = 0; q < N / 4; ++q) {
#pragma unroll
        for (int i = 0; i < 4; ++i) out[i] = q == 0 ? t.c[q][i] * h[q][i] : fmaf(t.c[q][i], h[q][i], out[i]);
      }
    }
    if constexpr (!OUTPUT) sum += d;
    return (out[0] + out[1]) + (out[2] + out[3]);
  };

  // The values of a group of rows, loaded a group ahead (rows past the chunk: the last one's again)
  struct Group { T u[kGroup], delta[kGroup], z[OUTPUT && G == 1 ? kGroup : 1]; };
  const auto load_group = [&](int32_t row) {
    Group g;
#pragma unroll
    for (int r = 0; r < kGroup; ++r) {
      const uint32_t at = uint32_t(min(row + r, rows.end - 1) - rows.begin) * pitch;
      g.u[r] = load_element<T>(ru, at_lane, at);
      g.delta[r] = load_element<T>(rd, at_lane, at);
      if constexpr (OUTPUT && G == 1) g.z[r] = load_element<T>(rz, at_lane, at);
    }
    return g;
  };
  // B and C of a tile of rows, by way of registers into one of the two buffers
  T staged_b[kPer], staged_c[OUTPUT ? kPer : 1];   // (past the chunk's rows or the states: zeros)
  const auto load_tile = [&](int32_t tile) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = int(threadIdx.x) + i * kThreads, r = e / kStates, n = e % kStates;
      const uint32_t at = n < a.dstate ? uint32_t(tile - rows.begin + r) * row_bytes + uint32_t(n) * sizeof(T) : kOutOfRange;
      staged_b[i] = load_element<T>(rB, at, 0);
      if constexpr (OUTPUT) staged_c[i] = load_element<T>(rC, at, 0);
    }
  };
  const auto put_tile = [&](int buffer) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = int(threadIdx.x) + i * kThreads, r = e / kStates, n = e % kStates;
      if (r < kRows) {
        Bs[buffer][r][n / N][n % 4][n % N / 4] = to_f32(staged_b[i]);
        if constexpr (OUTPUT) Cs[buffer][r][n] = to_f32(staged_c[i]);
      }
    }
  };
  // with G waves to a channel: the sum of a tile's parts, and y
  const auto join = [&](int32_t tile, uint32_t walked) {
    const int32_t cj = block_channel + int32_t(threadIdx.x) % kChannels;
    if (cj >= a.channels) return;
    const float skip_j = a.D != nullptr ? a.D[cj] : 0.f;
    for (int r = int(threadIdx.x) / kChannels; r < kRows; r += G) {
      if (!(walked >> r & 1u)) continue;
      const uint32_t at = uint32_t(tile + r - rows.begin) * pitch + uint32_t(cj) * sizeof(T);
      float out = skip_j * to_f32(load_element<T>(ru, at, 0));
#pragma unroll
      for (int g = 0; g < G; ++g) out += parts[r][g][int(threadIdx.x) % kChannels];
      if (has_z) out *= silu<EXACT>(to_f32(load_element<T>(rz, at, 0)));
      store_element(ry, at, 0, from_f32<T>(out));
    }
  };
  bool inside = s < a.seq.sequences && span.begin <= from && from < span.end;
  if (inside) enter(from);
  load_tile(from);
  put_tile(0);
  Group ahead = load_group(from);
  int buffer = 0;
  for (int32_t tile = from; tile < rows.end; tile += kRows, buffer ^= 1) {
    __syncthreads();   // the tile is in LDS, and the buffer of the one before is free
    const bool more = tile + kRows < rows.end;
    if (more) load_tile(tile + kRows);
    uint32_t walked = 0;   // the tile's rows that are in a sequence
#pragma unroll 1
    for (int part = 0; part < kRows && tile + part < rows.end; part += kGroup) {
      const int32_t row0 = tile + part;
      const Group now = ahead;
      if (row0 + kGroup < rows.end) ahead = load_group(row0 + kGroup);
      float d[kGroup], v[kGroup], gate[OUTPUT ? kGroup : 1];
#pragma unroll
      for (int r = 0; r < kGroup; ++r) {
        v[r] = to_f32(now.u[r]);
        d[r] = to_f32(now.delta[r]) + bias;
        if constexpr (OUTPUT) gate[r] = 1.f;
      }
      if (a.softplus) {
#pragma unroll
        for (int r = 0; r < kGroup; ++r) d[r] = softplus<EXACT>(d[r]);
      }
      if constexpr (OUTPUT && G == 1) {
        if (has_z) {
#pragma unroll
          for (int r = 0; r < kGroup; ++r) gate[r] = silu<EXACT>(to_f32(now.z[r]));
        }
      }
      const auto row_of = [&](int r, float dr, float vr, float gr, const Row& t) __attribute__((always_inline)) {
        const float read = token(dr, vr, t);
        if constexpr (OUTPUT && G == 1)
          store_element(ry, store_lane, uint32_t(row0 + r - rows.begin) * pitch, from_f32<T>(fmaf(skip, vr, read) * gr));
        if constexpr (OUTPUT && G > 1) parts[part + r][group][wave / G * kWave + lane] = read;
      };
      if (inside && row0 + kGroup <= min(span.end, rows.end)) {
        Row t = read_row(buffer, part);
#pragma unroll
        for (int r = 0; r < kGroup; ++r) {
          const Row next = read_row(buffer, part + (r + 1 < kGroup ? r + 1 : r));
          row_of(r, d[r], v[r], gate[OUTPUT ? r : 0], t);
          t = next;
        }
        walked |= ((1u << kGroup) - 1u) << part;
        if (row0 + kGroup == span.end) leave();
        continue;
      }
#pragma unroll 1
      for (int r = 0; r < kGroup && row0 + r < rows.end; ++r) {   // where sequences begin or end
        const int32_t row = row0 + r;
        if (OUTPUT && s < a.seq.sequences && span.end <= row) {   // (else all rows from `from` on are of one)
          a.seq.advance(row, s, span);
          inside = false;
        }
        if (s >= a.seq.sequences || row < span.begin) continue;
        if (!inside) {
          enter(row);
          inside = true;
        }
        float dr = d[0], vr = v[0], gr = gate[0];
#pragma unroll
        for (int i = 1; i < kGroup; ++i) {
          dr = r == i ? d[i] : dr;
          vr = r == i ? v[i] : vr;
          if constexpr (OUTPUT) gr = r == i ? gate[i] : gr;
        }
        row_of(r, dr, vr, gr, read_row(buffer, part + r));
        walked |= 1u << (part + r);
        if (row + 1 == span.end) leave();
      }
    }
    if constexpr (OUTPUT && G > 1) {
      __syncthreads();
      join(tile, walked);
    }
    if (more) put_tile(buffer ^ 1);
  }
  if constexpr (!OUTPUT) {
    if (!live) return;
#pragma unroll
    for (int n = 0; n < N; ++n)
      if (first_state + n < a.dstate)
        a.states[(int64_t(k) * a.dstate + first_state + n) * a.channels + c] = h[n / 4][n % 4];
    if (group == 0) a.sums[int64_t(k) * a.channels + c] = sum;
  }
}

// The value of lane `from` of every four neighbouring lanes, in all of them; that of the lane whose number differs in bit 0
// or in bit 1.
__device__ __forceinline__ float of_lane(float v, int from) {
  const int i = __float_as_int(v);
  switch (from) {
    case 0: return __int_as_float(__builtin_amdgcn_mov_dpp(i, 0x00, 0xF, 0xF, true));
    case 1: return __int_as_float(__builtin_amdgcn_mov_dpp(i, 0x55, 0xF, 0xF, true));
    case 2: return __int_as_float(__builtin_amdgcn_mov_dpp(i, 0xAA, 0xF, 0xF, true));
    default: return __int_as_float(__builtin_amdgcn_mov_dpp(i, 0xFF, 0xF, 0xF, true));
  }
}
__device__ __forceinline__ float other_of_pair(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0xB1, 0xF, 0xF, true));
}
__device__ __forceinline__ float other_pair(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x4E, 0xF, 0xF, true));
}

// Dense sequences walked whole by four lanes a channel, N states each.  Of four rows each of the lanes loads one, forms its
// step size and its gate, and writes its y; the step sizes go round as lane exchanges within the products that take them.
// Values and the next 16 rows of B and C are loaded a tile ahead: a SIMD may have one wave only (4 x 2048 x 4096 x 16: 109
// ns a row for one wave a SIMD, 72 a wave for four).
template <typename T, int N>
__global__ void __launch_bounds__(kThreads, 2) quad_kernel(ScanKernelArgs a) {
  constexpr bool EXACT = sizeof(T) == 4;
  constexpr int kStates = 4 * N, kGroups = kRows / 4;
  constexpr int kPer = (kRows * kStates + kThreads - 1) / kThreads;   // values of B, and of C, that a thread stages
  __shared__ __attribute__((aligned(16))) float Bs[2][kRows][kStates], Cs[2][kRows][kStates];
  const int lane = int(threadIdx.x) % kWave, q = lane % 4, first_state = q * N;
  const int32_t c = int32_t(blockIdx.y) * (kThreads / 4) + int32_t(threadIdx.x) / 4;
  const bool live = c < a.channels;
  const int32_t cc = min(c, a.channels - 1);   // lanes past the last channel compute it too and store nothing
  const int32_t s = int32_t(blockIdx.x), length = int32_t(a.seq.length.d);
  const int64_t base = int64_t(s) * length;
  float A2[N], h[N] = {};
  load_states<N>(a.A + int64_t(cc) * a.dstate, 1, first_state, a.dstate, A2);
  if (a.h0 != nullptr) load_states<N>(a.h0 + (int64_t(s) * a.channels + cc) * a.dstate, 1, first_state, a.dstate, h);
#pragma unroll
  for (int n = 0; n < N; ++n) A2[n] *= kLog2e;
  const float bias = a.delta_bias != nullptr ? a.delta_bias[cc] : 0.f, skip = a.D != nullptr ? a.D[cc] : 0.f;
  const bool has_z = a.z != nullptr;
  const uint32_t pitch = uint32_t(a.channels) * sizeof(T), bytes = uint32_t(length) * pitch;
  const uint32_t at_lane = uint32_t(q) * pitch + uint32_t(cc) * sizeof(T);
  const Rsrc ru = make_rsrc(static_cast<const T*>(a.u) + base * a.channels, bytes);
  const Rsrc rd = make_rsrc(static_cast<const T*>(a.delta) + base * a.channels, bytes);
  const Rsrc rz = make_rsrc(static_cast<const T*>(has_z ? a.z : a.u) + base * a.channels, bytes);
  const Rsrc ry = make_rsrc(static_cast<T*>(a.y) + base * a.channels, bytes);
  const uint32_t row_bytes = uint32_t(a.dstate) * sizeof(T), bc_bytes = uint32_t(length) * row_bytes;
  const Rsrc rB = make_rsrc(static_cast<const T*>(a.B) + base * a.dstate, bc_bytes);
  const Rsrc rC = make_rsrc(static_cast<const T*>(a.C) + base * a.dstate, bc_bytes);

  // what a lane needs of a tile of rows, loaded a tile ahead (rows past the sequence load as zero)
  struct Tile { T u[kGroups], delta[kGroups], z[kGroups]; };
  const auto load_values = [&](int32_t tile) {
    Tile t;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const uint32_t at = at_lane + uint32_t(tile + 4 * g) * pitch;
      t.u[g] = load_element<T>(ru, at, 0);
      t.delta[g] = load_element<T>(rd, at, 0);
      t.z[g] = load_element<T>(rz, at, 0);
    }
    return t;
  };
  T staged_b[kPer], staged_c[kPer];
  const auto load_tile = [&](int32_t tile) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = int(threadIdx.x) + i * kThreads, r = e / kStates, n = e % kStates;
      const uint32_t at = n < a.dstate ? uint32_t(tile + r) * row_bytes + uint32_t(n) * sizeof(T) : kOutOfRange;
      staged_b[i] = load_element<T>(rB, at, 0);
      staged_c[i] = load_element<T>(rC, at, 0);
    }
  };
  const auto put_tile = [&](int buffer) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = int(threadIdx.x) + i * kThreads, r = e / kStates, n = e % kStates;
      if (r < kRows) {
        Bs[buffer][r][n] = to_f32(staged_b[i]);
        Cs[buffer][r][n] = to_f32(staged_c[i]);
      }
    }
  };
  // a row of B and C, the lane's states
  struct Row { float b[N], c[N]; };
  const auto read_row = [&](int buffer, int r) __attribute__((always_inline)) {
    Row t;
    __builtin_memcpy(t.b, __builtin_assume_aligned(&Bs[buffer][r][first_state], N == 2 ? 8 : 16), sizeof(t.b));
    __builtin_memcpy(t.c, __builtin_assume_aligned(&Cs[buffer][r][first_state], N == 2 ? 8 : 16), sizeof(t.c));
    return t;
  };
  // one token: d its step size, dv that times u; returns the lane's part of C . h
  const auto token = [&](float d, float dv, const Row& t) __attribute__((always_inline)) {
    float out = 0.f;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      h[n] = fmaf(__builtin_amdgcn_exp2f(d * A2[n]), h[n], dv * t.b[n]);
      out = n == 0 ? t.c[0] * h[0] : fmaf(t.c[n], h[n], out);
    }
    return out;
  };
  struct Step { float d, dv, v, gate; };   // of the lane's row
  const auto prepare = [&](const Tile& t, int g) __attribute__((always_inline)) {
    Step p;
    p.v = to_f32(t.u[g]);
    const float raw = to_f32(t.delta[g]) + bias, soft = softplus<EXACT>(raw), open = silu<EXACT>(to_f32(t.z[g]));
    p.d = a.softplus ? soft : raw;
    p.dv = p.d * p.v;
    p.gate = has_z ? open : 1.f;
    return p;
  };
  // y of four rows: lane q gets row q's sum over the four lanes
  const auto finish = [&](const float (&out)[4], const Step& p, int32_t row0) __attribute__((always_inline)) {
    const bool odd = q & 1, high = q & 2;
    const float low_rows = (odd ? out[1] : out[0]) + other_of_pair(odd ? out[0] : out[1]);
    const float high_rows = (odd ? out[3] : out[2]) + other_of_pair(odd ? out[2] : out[3]);
    const float read = (high ? high_rows : low_rows) + other_pair(high ? low_rows : high_rows);
    const uint32_t at = live ? at_lane + uint32_t(row0) * pitch : kOutOfRange;
    store_element(ry, at, 0, from_f32<T>(fmaf(skip, p.v, read) * p.gate));
  };

  load_tile(0);
  Tile ahead = load_values(0);
  put_tile(0);
  int buffer = 0;
  for (int32_t tile = 0; tile < length; tile += kRows, buffer ^= 1) {
    __syncthreads();   // the tile is in LDS, and the buffer of the one before is free
    const bool more = tile + kRows < length;
    const Tile now = ahead;
    if (more) {
      load_tile(tile + kRows);
      ahead = load_values(tile + kRows);
    }
    if (tile + kRows <= length) {
      Step p = prepare(now, 0);
      Row t = read_row(buffer, 0);
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const Step next_p = prepare(now, g + 1 < kGroups ? g + 1 : g);
        float out[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const Row next = read_row(buffer, 4 * g + r + 1 < kRows ? 4 * g + r + 1 : 0);
          out[r] = token(of_lane(p.d, r), of_lane(p.dv, r), t);
          t = next;
        }
        finish(out, p, tile + 4 * g);
        p = next_p;
      }
    } else {
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const int32_t row0 = tile + 4 * g;
        if (row0 >= length) break;
        const Step p = prepare(now, g);
        float out[4] = {};
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (row0 + r < length) out[r] = token(of_lane(p.d, r), of_lane(p.dv, r), read_row(buffer, 4 * g + r));
        finish(out, p, row0);
      }
    }
    if (more) put_tile(buffer ^ 1);
  }
  if (!live || a.h_final == nullptr) return;
#pragma unroll
  for (int n = 0; n < N; ++n)
    if (first_state + n < a.dstate)
      a.h_final[(int64_t(s) * a.channels + c) * a.dstate + first_state + n] = h[n];
}

constexpr int kCarried = 16;

// chunk by chunk along every chain (a dense sequence, or all packed rows), one thread per channel and state.  Bound by
// the latency of its loads, of which 16 chunks' are under way at a time (16384 x 5120 16 us).
__global__ void __launch_bounds__(kThreads) carry_kernel(ScanKernelArgs a) {
  const int32_t c = int32_t(blockIdx.x) * kThreads + int32_t(threadIdx.x);
  const int32_t n = int32_t(blockIdx.y);
  if (c >= a.channels) return;
  const float A2 = a.A[int64_t(c) * a.dstate + n] * kLog2e;
  for (int32_t first = int32_t(blockIdx.z) * a.per_sequence; first < a.chunks;
       first += int32_t(gridDim.z) * a.per_sequence) {
    const int32_t last = first + a.per_sequence - 1;   // nothing enters a chain's first chunk; nothing reads its last's
    const int64_t pitch = int64_t(a.dstate) * a.channels;
    float* at = a.states + (int64_t(first) * a.dstate + n) * a.channels + c;
    struct Group { float own[kCarried], sum[kCarried]; int32_t reset[kCarried]; };
    const auto load = [&](int32_t k) {   // (past the last: its values again)
      Group g;
#pragma unroll
      for (int i = 0; i < kCarried; ++i) {
        const int32_t j = min(k + i, last - 1);
        g.own[i] = at[(j - first) * pitch];
        g.sum[i] = a.sums[int64_t(j) * a.channels + c];
        g.reset[i] = a.resets[j];
      }
      return g;
    };
    float h = 0.f;
    Group ahead = load(first);
    for (int32_t k = first; k < last; k += kCarried) {   // the loads of one group of chunks ahead of the other's sums
      const Group now = ahead;
      if (k + kCarried < last) ahead = load(k + kCarried);
#pragma unroll
      for (int i = 0; i < kCarried; ++i) {
        h = now.reset[i] ? now.own[i] : fmaf(__builtin_amdgcn_exp2f(now.sum[i] * A2), h, now.own[i]);
        if (k + i < last) at[(k + i - first) * pitch] = h;
      }
    }
  }
}

// Up to four neighbouring elements at any alignment; those past `count` are 0.
template <typename T>
__device__ __forceinline__ void load_four(const T* __restrict__ p, int count, float (&v)[4]) {
  struct { T e[4]; } raw = {};
  if (count >= 4) {
    __builtin_memcpy(&raw, p, sizeof(raw));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < count) raw.e[i] = p[i];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = to_f32(raw.e[i]);
}

// One token for every sequence.  HBM-bound by the states (256 x 8192 x 16: 55 us, 4.9 TB/s): `lanes` neighbouring lanes
// take a channel, four states each, and K sequences one after another, whose loads are all under way together and share
// A (109 us with one sequence a lane).
template <typename T, int K>
__global__ void __launch_bounds__(kThreads) step_kernel(float* __restrict__ state, const T* __restrict__ u,
                                                        const T* __restrict__ delta, const float* __restrict__ A,
                                                        const T* __restrict__ B, const T* __restrict__ C,
                                                        const float* __restrict__ D, const T* __restrict__ z,
                                                        const float* __restrict__ delta_bias, T* __restrict__ y,
                                                        int32_t batch, int32_t channels, int32_t dstate, int32_t lanes,
                                                        int32_t channel_blocks, bool use_softplus) {
  constexpr bool EXACT = sizeof(T) == 4;
  const int32_t s0 = int32_t(blockIdx.x) / channel_blocks * K;
  const int32_t c0 = int32_t(blockIdx.x) % channel_blocks * (kThreads / lanes) + int32_t(threadIdx.x) / lanes;
  const bool live = c0 < channels;   // (all lanes of a channel are, or none: the others keep the sums' lanes filled)
  const int32_t c = min(c0, channels - 1);
  const int first = int(threadIdx.x) % lanes * 4, count = dstate - first;
  float a[4], h[K][4], b[K][4], cs[K][4], d[K], v[K], gate[K];
  load_four(A + int64_t(c) * dstate + first, count, a);
  const float bias = delta_bias != nullptr ? delta_bias[c] : 0.f, skip = D != nullptr ? D[c] : 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int64_t s = min(s0 + k, batch - 1), at = s * channels + c;
    load_four(state + at * dstate + first, count, h[k]);
    d[k] = to_f32(delta[at]) + bias;
    v[k] = to_f32(u[at]);
    gate[k] = z != nullptr ? to_f32(z[at]) : 0.f;
    load_four(B + s * dstate + first, count, b[k]);
    load_four(C + s * dstate + first, count, cs[k]);
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (s0 + k >= batch) break;
    const int64_t at = int64_t(s0 + k) * channels + c;
    if (use_softplus) d[k] = softplus<EXACT>(d[k]);
    float out = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h[k][i] = fmaf(__builtin_amdgcn_exp2f(d[k] * a[i] * kLog2e), h[k][i], d[k] * v[k] * b[k][i]);
      out = i < count ? fmaf(cs[k][i], h[k][i], out) : out;
    }
    if (live) {
      float* to = state + at * dstate + first;
      if (count >= 4) {
        __builtin_memcpy(to, h[k], 16);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < count) to[i] = h[k][i];
      }
    }
    for (int n = 1; n < lanes; n <<= 1) out += __shfl_xor(out, n);
    out = fmaf(skip, v[k], out);
    if (z != nullptr) out *= silu<EXACT>(gate[k]);
    if (live && first == 0) y[at] = from_f32<T>(out);
  }
}

// ---- host ----

struct Plan {
  bool quad;   // quad_kernel: sequences are the chunks
  int32_t chunk, per_sequence, chunks;
  size_t sums, resets, bytes;   // byte offsets behind the states, and the total
};

constexpr int64_t kSimds = 1024;   // of a whole chip; the workspace's size does not depend on the device

constexpr int state_groups(int32_t dstate) { return dstate <= 16 ? 1 : dstate <= 32 ? 2 : 4; }

// Microseconds by both ways, for up to 8, 16, 32 and 64 states.  quad_kernel: a row takes `row` and `wave` more for every
// wave that a SIMD holds.  Chunks: kLaunches for three kernels, and `work` for a row of 16 x 1024 channels.  Measured, quad
// and chunks: 2048 x 4096 x 16 states with 2 sequences 219 and 144, with 4 223 and 257, with 8 344 and 467; 1 x 128 x 4096
// 17 and 28, 1 x 512 x 8192 58 and 64, 1001 x 1024 110 and 34; 2 x 2048 x 4096 with 8 states 164 and 94, with 32 332 and
// 304, with 64 531 and 537.
struct Costs { double row, wave, work; };
constexpr Costs kCosts[] = {{0.036, 0.046, 0.080}, {0.050, 0.058, 0.115}, {0.076, 0.088, 0.28}, {0.100, 0.165, 0.52}};
constexpr double kLaunches = 25.;

bool quads_win(int64_t length, int64_t chains, int32_t channels, int32_t dstate) {
  const Costs& c = kCosts[dstate <= 8 ? 0 : dstate <= 16 ? 1 : dstate <= 32 ? 2 : 3];
  const int64_t waves = chains * ((int64_t(channels) + 15) / 16);
  const double quad = double(length) * (c.row + c.wave * double((waves + kSimds - 1) / kSimds));
  return quad <= kLaunches + double(length) * double(waves) / kSimds * c.work;
}

// Which way, and how long a chunk is: as many chunks as fill the three waves that a SIMD holds a whole number of times; a
// chunk has 16 to 256 rows (carried states are traffic, and the sum of d is kept precise).
bool make_plan(int32_t sequences, int64_t tokens, int32_t channels, int32_t dstate, bool packed, Plan* p) {
  const int64_t length = packed ? tokens : tokens / sequences, chains = packed ? 1 : sequences;
  // a sequence's rows are addressed in 32 bits
  p->quad = !packed && length > 0 && length * std::max(channels, dstate) < int64_t(1) << 29 &&
            quads_win(length, chains, channels, dstate);
  int64_t chunk = std::max<int64_t>(length, 1);
  if (!p->quad) {
    const int64_t waves = chains * ((int64_t(channels) + kWave - 1) / kWave) * state_groups(dstate);
    const int64_t least = (length + 255) / 256, rounds = (least * waves + 3 * kSimds - 1) / (3 * kSimds);
    const int64_t number = std::max(least, rounds * 3 * kSimds / waves);
    chunk = number > 0 ? (length + number - 1) / number : 1;
    chunk = std::min<int64_t>(256, std::max<int64_t>(16, (chunk + kGroup - 1) / kGroup * kGroup));
  }
  const int64_t per = (length + chunk - 1) / chunk, chunks = per * chains;
  if (chunks >= int64_t(1) << 23) return false;   // a grid's threads along x in 32 bits
  p->chunk = int32_t(chunk);
  p->per_sequence = int32_t(per);
  p->chunks = int32_t(chunks);
  const double need = double(chunks) * channels * (dstate + 1) * 4.0;
  if (need >= double(int64_t(1) << 40)) return false;
  const auto round = [](size_t n) { return (n + 255) & ~size_t(255); };
  const size_t carried = per > 1 ? size_t(chunks) : 0;
  p->sums = round(carried * dstate * channels * 4);
  p->resets = p->sums + round(carried * channels * 4);
  p->bytes = std::max<size_t>(256, p->resets + round(carried * 4));
  return true;
}

template <typename T, int N, int G>
hipError_t launch_states(const ScanKernelArgs& a, hipStream_t stream) {
  const uint32_t blocks = uint32_t((a.channels + kThreads / G - 1) / (kThreads / G));
  // grid.x: the chunks, and where sequences may have no rows some blocks that look for those, at up to 64 sequences each
  // (2^20 of them with 16 states, 5 channels: 48 ms by 64 blocks in all)
  const bool empty = a.h_final != nullptr && (a.seq.offsets != nullptr || a.seq.tokens == 0);
  const uint32_t extra = empty ? uint32_t(std::min(a.seq.sequences, std::max(64, a.seq.sequences / 64))) : 0u;
  if (a.per_sequence > 1) {
    chunk_kernel<T, N, G, false><<<dim3(a.chunks, blocks), kThreads, 0, stream>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const uint32_t chains = uint32_t(std::min(a.chunks / a.per_sequence, 32768));
    carry_kernel<<<dim3((a.channels + kThreads - 1) / kThreads, a.dstate, chains), kThreads, 0, stream>>>(a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.chunks + extra == 0) return hipSuccess;
  chunk_kernel<T, N, G, true><<<dim3(a.chunks + extra, blocks), kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

template <typename T, int N>
hipError_t launch_quad(const ScanKernelArgs& a, hipStream_t stream) {
  quad_kernel<T, N><<<dim3(a.seq.sequences, (a.channels + kThreads / 4 - 1) / (kThreads / 4)), kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_scan(const ScanKernelArgs& a, bool quad, hipStream_t stream) {
  if (quad) {
    if (a.dstate <= 8) return launch_quad<T, 2>(a, stream);
    switch (state_groups(a.dstate)) {
      case 1: return launch_quad<T, 4>(a, stream);
      case 2: return launch_quad<T, 8>(a, stream);
      default: return launch_quad<T, 16>(a, stream);
    }
  }
  if (a.dstate <= 8) return launch_states<T, 8, 1>(a, stream);
  switch (state_groups(a.dstate)) {
    case 1: return launch_states<T, 16, 1>(a, stream);
    case 2: return launch_states<T, 16, 2>(a, stream);
    default: return launch_states<T, 16, 4>(a, stream);
  }
}

int32_t step_lanes(int32_t dstate) {   // of a channel, with four states each
  int32_t lanes = 1;
  while (lanes * 4 < dstate) lanes *= 2;
  return lanes;
}
int32_t step_channel_blocks(int32_t channels, int32_t lanes) { return (channels + kThreads / lanes - 1) / (kThreads / lanes); }

template <typename T>
hipError_t launch_step(float* state, const void* u, const void* delta, const float* A, const void* B, const void* C,
                       const float* D, const void* z, const float* delta_bias, void* y, int32_t batch, int32_t channels,
                       int32_t dstate, bool softplus, hipStream_t stream) {
  const int32_t lanes = step_lanes(dstate), channel_blocks = step_channel_blocks(channels, lanes);
  const bool many = selective_step_plan(batch, channels, dstate) == 4;
  const int64_t blocks = int64_t(channel_blocks) * (many ? (batch + 3) / 4 : batch);
  const dim3 grid = dim3(uint32_t(blocks));
  const T *in = static_cast<const T*>(u), *steps = static_cast<const T*>(delta), *gate = static_cast<const T*>(z);
  const T *b = static_cast<const T*>(B), *c = static_cast<const T*>(C);
  const auto kernel = many ? step_kernel<T, 4> : step_kernel<T, 1>;
  kernel<<<grid, kThreads, 0, stream>>>(state, in, steps, A, b, c, D, gate, delta_bias, static_cast<T*>(y), batch, channels,
                                        dstate, lanes, channel_blocks, softplus);
  return hipGetLastError();
}

}  // namespace

size_t selective_workspace_bytes(int32_t sequences, int64_t tokens, int32_t channels, int32_t dstate, bool packed) {
  Plan p;
  return make_plan(sequences, tokens, channels, dstate, packed, &p) ? p.bytes : 0;
}

int32_t selective_scan_plan(int32_t sequences, int64_t tokens, int32_t channels, int32_t dstate, bool packed) {
  Plan p;
  if (!make_plan(sequences, tokens, channels, dstate, packed, &p)) return -1;
  return p.quad ? 0 : p.chunk;
}

// four sequences a lane once they leave a block for every compute unit
int32_t selective_step_plan(int32_t batch, int32_t channels, int32_t dstate) {
  return int64_t(step_channel_blocks(channels, step_lanes(dstate))) * (batch / 4) >= 256 ? 4 : 1;
}

hipError_t launch_selective_scan(const SelectiveArgs& s, hipStream_t stream) {
  Plan p;
  if (!make_plan(s.sequences, s.tokens, s.channels, s.dstate, s.offsets != nullptr, &p)) return hipErrorInvalidValue;
  ScanKernelArgs a = {};
  a.seq = make_sequences(s.offsets, s.sequences, s.tokens);
  a.u = s.u;
  a.delta = s.delta;
  a.A = s.A;
  a.B = s.B;
  a.C = s.C;
  a.D = s.D;
  a.z = s.z;
  a.delta_bias = s.delta_bias;
  a.h0 = s.h0;
  a.y = s.y;
  a.h_final = s.h_final;
  char* base = static_cast<char*>(s.workspace);
  a.states = reinterpret_cast<float*>(base);
  a.sums = reinterpret_cast<float*>(base + p.sums);
  a.resets = reinterpret_cast<int32_t*>(base + p.resets);
  a.channels = s.channels;
  a.dstate = s.dstate;
  a.chunk = p.chunk;
  a.per_sequence = p.per_sequence;
  a.chunks = p.chunks;
  a.softplus = s.softplus;
  switch (s.dtype) {
    case SSDQ_DTYPE_F32: return launch_scan<float>(a, p.quad, stream);
    case SSDQ_DTYPE_F16: return launch_scan<_Float16>(a, p.quad, stream);
    default: return launch_scan<__bf16>(a, p.quad, stream);
  }
}

hipError_t launch_selective_step(int32_t dtype, float* state, const void* u, const void* delta, const float* A,
                                 const void* B, const void* C, const float* D, const void* z, const float* delta_bias,
                                 void* y, int32_t batch, int32_t channels, int32_t dstate, bool softplus,
                                 hipStream_t stream) {
  switch (dtype) {
    case SSDQ_DTYPE_F32:
      return launch_step<float>(state, u, delta, A, B, C, D, z, delta_bias, y, batch, channels, dstate, softplus, stream);
    case SSDQ_DTYPE_F16:
      return launch_step<_Float16>(state, u, delta, A, B, C, D, z, delta_bias, y, batch, channels, dstate, softplus, stream);
    default:
      return launch_step<__bf16>(state, u, delta, A, B, C, D, z, delta_bias, y, batch, channels, dstate, softplus, stream);
  }
}

}  // namespace ssdq
