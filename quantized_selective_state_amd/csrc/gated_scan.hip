// Gated linear recurrence h_t = a_t h_{t-1} + b_t with a gate per channel, its gradient and its
// single-token step (Ternary Mamba, Section 1, states the recurrence).
//
// The maps h -> A h + H compose associatively, (A2, H2) o (A1, H1) = (A2 A1, A2 H1 + H2), so a
// sequence is cut into tiles of 256 tokens x 64 channels.  A block of 256 threads holds one tile in
// registers: a thread has V neighbouring channels (16 bytes where the row length allows) of 64 / V
// consecutive tokens.  It composes its tokens' maps, the maps are scanned over the threads of a wave
// and the block's waves, the tile's map is published, and the state entering the tile is joined from
// the maps of the tiles before it; then each thread runs its tokens once more from its entering state
// and stores.  Every input is read from memory once and every output written once.
//
// The gradient's recurrence k_t = a_t (dh_t + k_{t+1}) is the same scan from a sequence's end with the
// maps (a_t, a_t dh_t), so both directions share the code below.
#include "gated_types.h"

namespace ssdq {
namespace {

constexpr int kBlock = SSDQ_CHECKPOINT_BLOCK;   // channels of a tile, and of a checkpoint's scale
constexpr int kRows = 256;                      // tokens of a tile
constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kPerThread = kRows * kBlock / kThreads;   // elements of each tensor a thread holds

// Tiles of a sequence are joined in groups: a tile reads the maps of the tiles of its group before
// it, and of the group before that only the last tile's, which publishes the state it ended with as
// the map (0, state) once it knows that; so does a sequence's first tile.  This fixes the order of every
// product and sum (the same bits on every run) and bounds what a tile reads (16 maps) whatever the length.
constexpr int kGroup = 16;

// Workspace: a ticket counter and the tiles' maps (A, H), in words that are all ones until
// published.  A published word is never all ones: A = NaN is stored with one fixed image.
constexpr size_t kTicketBytes = 256;
constexpr uint64_t kNoMap = ~uint64_t(0);
constexpr int kMostPolls = 1 << 24;   // far beyond any wait; a state is NaN if it is ever reached

struct Plan {
  int32_t tiles;        // most tiles of the call
  int32_t chans;        // channel tiles
  int32_t per_sequence; // dense: tiles of a sequence (0: packed)
  bool single;          // every sequence is one tile: nothing is published
  uint64_t* maps;       // (tiles, chans * 64)
  uint32_t* ticket;
};

// Whole sequences: tiles of the call and whether each sequence fits one.
bool plan_sizes(int32_t sequences, int64_t tokens, int32_t channels, bool packed, Plan* p) {
  if (channels > (1 << 20)) return false;   // a tile's byte offsets stay below 2^31
  p->chans = (channels + kBlock - 1) / kBlock;
  int64_t tiles;
  if (packed) {
    p->per_sequence = 0;
    p->single = tokens <= kRows;
    tiles = p->single ? sequences : tokens / kRows + sequences;
  } else {
    const int64_t len = tokens / sequences;
    const int64_t per = len <= kRows ? 1 : (len + kRows - 1) / kRows;
    p->single = per == 1;
    tiles = per * sequences;
    p->per_sequence = int32_t(per);
  }
  // a grid holds fewer than 2^32 threads
  if (tiles * p->chans >= (int64_t(1) << 24)) return false;
  p->tiles = int32_t(tiles);
  return true;
}

size_t map_bytes(const Plan& p) { return size_t(p.tiles) * p.chans * kBlock * sizeof(uint64_t); }

// Buffer accesses: out-of-range reads give zeros, out-of-range writes are dropped.
__device__ __forceinline__ void load_bytes(Rsrc r, uint32_t off, v4u& v) { v = __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0); }
__device__ __forceinline__ void load_bytes(Rsrc r, uint32_t off, v2u& v) { v = __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0); }
__device__ __forceinline__ void load_bytes(Rsrc r, uint32_t off, uint32_t& v) { v = __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0); }
__device__ __forceinline__ void load_bytes(Rsrc r, uint32_t off, u16& v) { v = __builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0); }
__device__ __forceinline__ void load_bytes(Rsrc r, uint32_t off, uint8_t& v) { v = __builtin_amdgcn_raw_buffer_load_b8(r, off, 0, 0); }
__device__ __forceinline__ void store_bytes(Rsrc r, uint32_t off, v4u v) { __builtin_amdgcn_raw_buffer_store_b128(v, r, off, 0, 0); }
__device__ __forceinline__ void store_bytes(Rsrc r, uint32_t off, v2u v) { __builtin_amdgcn_raw_buffer_store_b64(v, r, off, 0, 0); }
__device__ __forceinline__ void store_bytes(Rsrc r, uint32_t off, uint32_t v) { __builtin_amdgcn_raw_buffer_store_b32(v, r, off, 0, 0); }
__device__ __forceinline__ void store_bytes(Rsrc r, uint32_t off, u16 v) { __builtin_amdgcn_raw_buffer_store_b16(v, r, off, 0, 0); }
__device__ __forceinline__ void store_bytes(Rsrc r, uint32_t off, uint8_t v) { __builtin_amdgcn_raw_buffer_store_b8(v, r, off, 0, 0); }

template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_pack(Rsrc r, uint32_t off) {
  Pack<T, V> p;
  load_bytes(r, off, p.raw);
  return p;
}
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> to_pack(const float (&x)[V]) {
  typename Pack<T, V>::Elements e;
#pragma unroll
  for (int v = 0; v < V; ++v) e.e[v] = from_f32<T>(x[v]);
  return Pack<T, V>{__builtin_bit_cast(typename Pack<T, V>::Raw, e)};
}

__device__ __forceinline__ uint64_t map_word(float A, float H) {
  const uint32_t a = A != A ? 0x7FC00000u : __float_as_uint(A);
  return uint64_t(a) | (uint64_t(__float_as_uint(H)) << 32);
}

// Relaxed device-scope accesses: a word carries its own validity, so nothing else is ordered by them.
__device__ __forceinline__ uint64_t peek(const uint64_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void publish(uint64_t* p, uint64_t v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The rows of sequence s; whatever the offsets hold, they stay inside the tensors.
__device__ __forceinline__ void sequence_rows(const GatedArgs& g, int s, int32_t& first, int32_t& last) {
  first = min(max(g.offsets[s], 0), int32_t(g.tokens));
  last = min(max(g.offsets[s + 1], first), int32_t(g.tokens));
}
__device__ __forceinline__ int32_t sequence_tiles(int32_t len) { return len <= kRows ? 1 : (len + kRows - 1) / kRows; }

struct Tile {
  int32_t seq;       // -1: no such tile
  int32_t chunk;     // tiles of the sequence before this one, in scan order
  int32_t chunks;    // tiles of the sequence
  int32_t base;      // index of the sequence's first tile in the workspace
  int32_t first;     // the sequence's rows
  int32_t len;
};

// Tile number i of a packed call: each thread counts the tiles of a run of sequences, a scan over the
// block finds the run that holds tile i, and its thread the sequence.
__device__ __forceinline__ Tile packed_tile(const GatedArgs& g, int32_t i, Tile* shared, int32_t* sums) {
  const int tid = int(threadIdx.x), lane = tid & 63, wave = tid >> 6;
  const int per = (g.sequences + kThreads - 1) / kThreads;
  const int s0 = min(tid * per, g.sequences), s1 = min(s0 + per, g.sequences);
  int32_t mine = 0;
  for (int s = s0; s < s1; ++s) {
    int32_t a, b;
    sequence_rows(g, s, a, b);
    mine += sequence_tiles(b - a);
  }
  int32_t upto = mine;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int32_t v = __shfl_up(upto, o, 64);
    if (lane >= o) upto += v;
  }
  if (lane == 63) sums[wave] = upto;
  if (tid == 0) shared->seq = -1;
  __syncthreads();
  int32_t before = upto - mine;
  for (int w = 0; w < wave; ++w) before += sums[w];
  if (i >= before && i < before + mine) {
    for (int s = s0; s < s1; ++s) {
      int32_t a, b;
      sequence_rows(g, s, a, b);
      const int32_t n = sequence_tiles(b - a);
      if (i < before + n) {
        *shared = Tile{s, i - before, n, before, a, b - a};
        break;
      }
      before += n;
    }
  }
  __syncthreads();
  return *shared;
}

// What the backward pass reads the saved states from, and what the forward pass writes
constexpr int kForward = 0, kForwardSave = 1, kBackward = 2, kBackwardSaved = 3;

template <typename T, int KIND, int V, int MODE>
__global__ void __launch_bounds__(kThreads) gated_kernel(GatedArgs g, Plan p) {
  constexpr bool kBack = MODE == kBackward || MODE == kBackwardSaved;
  constexpr int LPR = kBlock / V;        // lanes of a row
  constexpr int kGroups = kWave / LPR;   // runs of tokens in a wave
  constexpr int R = kPerThread / V;      // tokens of a run
  static_assert(kGroups * kWaves * R == kRows, "a block holds one tile");

  __shared__ float sA[kWaves][kBlock], sH[kWaves][kBlock], sIn[kBlock];
  __shared__ Tile sTile;
  __shared__ int32_t sSums[kWaves];
  __shared__ uint32_t sTicket;

  const int tid = int(threadIdx.x), lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  // Tiles are taken in the order in which blocks start, so that a tile's predecessors are always
  // held by blocks that run already; they publish before they wait for anything.
  uint32_t order = blockIdx.x;
  if (!p.single) {
    if (tid == 0) sTicket = __hip_atomic_fetch_add(p.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    order = __builtin_amdgcn_readfirstlane(sTicket);
  }
  const int32_t index = int32_t(order / uint32_t(p.chans));
  const int32_t blk = int32_t(order % uint32_t(p.chans));
  Tile t;
  if (p.per_sequence) {
    // dense: first tiles of all sequences, then their second ones, ...
    const int32_t len = int32_t(g.tokens / g.sequences);
    t.chunk = index / g.sequences;
    t.seq = index - t.chunk * g.sequences;
    t.chunks = p.per_sequence;
    t.base = t.seq * p.per_sequence;
    t.first = t.seq * len;
    t.len = len;
  } else {
    t = packed_tile(g, index, &sTile, sSums);
    t.seq = __builtin_amdgcn_readfirstlane(t.seq);
    if (t.seq < 0) return;
    t.chunk = __builtin_amdgcn_readfirstlane(t.chunk);
    t.chunks = __builtin_amdgcn_readfirstlane(t.chunks);
    t.base = __builtin_amdgcn_readfirstlane(t.base);
    t.first = __builtin_amdgcn_readfirstlane(t.first);
    t.len = __builtin_amdgcn_readfirstlane(t.len);
  }
  const int32_t nrows = min(kRows, t.len - t.chunk * kRows);
  // rows of the tile: the scan runs from the first to the last, or from the last to the first
  const int64_t row0 = kBack ? int64_t(t.first) + t.len - t.chunk * kRows - nrows : int64_t(t.first) + t.chunk * kRows;

  const int group = lane / LPR, col = (lane % LPR) * V;
  const int c = blk * kBlock + col;
  const bool in = c < g.channels;
  const uint32_t rowbytes = uint32_t(g.channels) * uint32_t(sizeof(T));
  const uint32_t tilebytes = uint32_t(nrows) * rowbytes;
  const int run = (wave * kGroups + group) * R;   // scan position of the run's first token
  // byte offset of scan position run + i in the tile: base + i * step; past the tile's rows it is out of
  // range (below zero it wraps to above 2^31), and so it is in every row for a lane past the channels
  const uint32_t base = !in ? kOutOfRange
                            : uint32_t(kBack ? nrows - 1 - run : run) * rowbytes + uint32_t(c) * uint32_t(sizeof(T));
  const uint32_t step = !in ? 0u : kBack ? 0u - rowbytes : rowbytes;
  const int64_t start = row0 * g.channels;

  const Rsrc rgate = make_rsrc(static_cast<const T*>(g.gate) + start, tilebytes);
  const Rsrc rsrc = make_rsrc(static_cast<const T*>(kBack ? g.dh : g.u) + start, tilebytes);
  typedef Pack<T, V> P;
  P pg[R], ps[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    pg[i] = load_pack<T, V>(rgate, base + uint32_t(i) * step);
    ps[i] = load_pack<T, V>(rsrc, base + uint32_t(i) * step);
  }
  // the states that the tokens start from are those of the row before; the sequence's first token
  // starts from h0, so its row is out of range
  P ph[R], pu[R];
  typedef Pack<int8_t, V> PC;
  PC pc[R];
  float sc[R];
  if constexpr (kBack) {
    const bool has_first = row0 == t.first;
    // position of the first token in this run, or none
    const int first_at = has_first ? nrows - 1 - run : -1;
    if constexpr (MODE == kBackward) {
      const Rsrc rh = make_rsrc(static_cast<const T*>(g.h) + (start - g.channels), tilebytes);
#pragma unroll
      for (int i = 0; i < R; ++i)
        ph[i] = load_pack<T, V>(rh, i == first_at ? kOutOfRange : base + uint32_t(i) * step);
    } else {
      const uint32_t crow = uint32_t(g.channels), srow = 4u * uint32_t(p.chans);
      const Rsrc rc = make_rsrc(g.codes + (start - g.channels), uint32_t(nrows) * crow);
      const Rsrc rs = make_rsrc(g.scale + (row0 - 1) * p.chans, uint32_t(nrows) * srow);
      const uint32_t cbase = in ? uint32_t(nrows - 1 - run) * crow + uint32_t(c) : kOutOfRange;
      const uint32_t cstep = in ? 0u - crow : 0u;
      const uint32_t sbase = uint32_t(nrows - 1 - run) * srow + 4u * uint32_t(blk);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        pc[i] = load_pack<int8_t, V>(rc, i == first_at ? kOutOfRange : cbase + uint32_t(i) * cstep);
        sc[i] = buf_loadf(rs, i == first_at ? kOutOfRange : sbase - uint32_t(i) * srow);
      }
    }
    if constexpr (KIND == SSDQ_GATE_LOGIT) {
      const Rsrc ru = make_rsrc(static_cast<const T*>(g.u) + start, tilebytes);
#pragma unroll
      for (int i = 0; i < R; ++i) pu[i] = load_pack<T, V>(ru, base + uint32_t(i) * step);
    }
  }

  // a run's map, token by token.  A row past the tile has gate and input 0: the identity for a log
  // gate, made the identity for a logit below.
  float a[R][V], b[R][V], cc[R][V];   // b: what a token adds (forward), dh (backward)
  float A[V], H[V];
#pragma unroll
  for (int v = 0; v < V; ++v) A[v] = 1.f, H[v] = 0.f;
#pragma unroll
  for (int i = 0; i < R; ++i) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float m;
      gate_terms<KIND>(pg[i][v], a[i][v], m);
      if constexpr (KIND == SSDQ_GATE_LOGIT) {
        if (run + i >= nrows) a[i][v] = 1.f;
        if constexpr (kBack) cc[i][v] = m;
      }
      b[i][v] = kBack || KIND == SSDQ_GATE_LOG ? ps[i][v] : m * ps[i][v];
      A[v] *= a[i][v];
      H[v] = kBack ? a[i][v] * (b[i][v] + H[v]) : fmaf(a[i][v], H[v], b[i][v]);
    }
  }

  // inclusive scan of the runs' maps within the wave, then each run's exclusive map
#pragma unroll
  for (int o = 1; o < kGroups; o <<= 1) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float pA = __shfl_up(A[v], o * LPR, 64), pH = __shfl_up(H[v], o * LPR, 64);
      if (group >= o) {
        H[v] = fmaf(A[v], pH, H[v]);
        A[v] *= pA;
      }
    }
  }
  if (group == kGroups - 1) {
#pragma unroll
    for (int v = 0; v < V; ++v) sA[wave][col + v] = A[v], sH[wave][col + v] = H[v];
  }
  if constexpr (kGroups > 1) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float pA = __shfl_up(A[v], LPR, 64), pH = __shfl_up(H[v], LPR, 64);
      A[v] = group ? pA : 1.f;
      H[v] = group ? pH : 0.f;
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) A[v] = 1.f, H[v] = 0.f;
  }
  __syncthreads();

  if (wave == 0) {
    // a lane per channel: the tile's map, and the state entering the tile
    const int64_t cpad = int64_t(p.chans) * kBlock, ch = int64_t(blk) * kBlock + lane;
    const bool some = ch < g.channels;
    const int64_t sat = int64_t(t.seq) * g.channels + ch;
    float tA = 1.f, tH = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      tH = fmaf(sA[w][lane], tH, sH[w][lane]);
      tA *= sA[w][lane];
    }
    const float* init = kBack ? g.dh_final : g.h0;
    const bool last = t.chunk == t.chunks - 1, ends_group = t.chunk % kGroup == kGroup - 1;
    uint64_t* maps = p.maps + int64_t(t.base) * cpad + ch;
    float x = 0.f;
    if (t.chunk == 0) {
      // only this tile reads the initial state (which the final one may overwrite)
      x = some && init ? init[sat] : 0.f;
    } else {
      if (!last && !ends_group) publish(maps + int64_t(t.chunk) * cpad, map_word(tA, tH));
      const int from = max(t.chunk / kGroup * kGroup - 1, 0), n = t.chunk - from;
      uint64_t got[kGroup];
      for (int polls = 0;; ++polls) {
        bool all = true;
#pragma unroll
        for (int j = 0; j < kGroup; ++j) {
          if (j < n) {
            got[j] = peek(maps + int64_t(from + j) * cpad);
            all = all && got[j] != kNoMap;
          }
        }
        if (__all(all) || polls == kMostPolls) break;
        __builtin_amdgcn_s_sleep(1);
      }
#pragma unroll
      for (int j = 0; j < kGroup; ++j)
        if (j < n) x = fmaf(__uint_as_float(uint32_t(got[j])), x, __uint_as_float(uint32_t(got[j] >> 32)));
    }
    sIn[lane] = x;
    const float end = fmaf(tA, x, tH);
    if (!last && (t.chunk == 0 || ends_group)) publish(maps + int64_t(t.chunk) * cpad, map_word(0.f, end));
    float* out = kBack ? g.dh0 : g.h_final;
    if (last && out && some) out[sat] = t.len ? end : x;
  }
  __syncthreads();

  // the state entering each run: the tile's, then the waves before, then the runs before
  float x[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float y = sIn[col + v];
    for (int w = 0; w < wave; ++w) y = fmaf(sA[w][col + v], y, sH[w][col + v]);
    x[v] = fmaf(A[v], y, H[v]);
  }

  if constexpr (!kBack) {
    const Rsrc rh = make_rsrc(static_cast<T*>(g.h) + start, tilebytes);
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
      for (int v = 0; v < V; ++v) x[v] = fmaf(a[i][v], x[v], b[i][v]);
      const P out = to_pack<T, V>(x);
      store_bytes(rh, base + uint32_t(i) * step, out.raw);
      if constexpr (MODE == kForwardSave) {
        uint32_t most = 0;
        if (in) {
#pragma unroll
          for (int v = 0; v < V; ++v) most = max(most, __float_as_uint(fabsf(out[v])));
        }
        const float s = checkpoint_scale(row_umax<LPR>(most));
        const uint32_t crow = uint32_t(g.channels), srow = 4u * uint32_t(p.chans);
        const Rsrc rc = make_rsrc(g.codes + start, uint32_t(nrows) * crow);
        const Rsrc rs = make_rsrc(g.scale + row0 * p.chans, uint32_t(nrows) * srow);
        store_bytes(rc, in ? uint32_t(run + i) * crow + uint32_t(c) : kOutOfRange,
                    codes_of<V>(out, s));
        store_bytes(rs, col == 0 ? uint32_t(run + i) * srow + 4u * uint32_t(blk) : kOutOfRange, __float_as_uint(s));
      }
    }
  } else {
    const Rsrc rdg = make_rsrc(static_cast<T*>(g.dgate) + start, tilebytes);
    const Rsrc rdu = make_rsrc(static_cast<T*>(g.du) + start, tilebytes);
    const int first_at = row0 == t.first ? nrows - 1 - run : -1;
    float h0[V];
#pragma unroll
    for (int v = 0; v < V; ++v) h0[v] = 0.f;
    if (g.h0 && in && first_at >= 0 && first_at < R) {
#pragma unroll
      for (int v = 0; v < V; ++v) h0[v] = g.h0[int64_t(t.seq) * g.channels + c + v];
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float dg[V], du[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float before;
        if constexpr (MODE == kBackward) before = ph[i][v];
        else before = pc[i][v] * sc[i];
        if (i == first_at) before = h0[v];
        const float d = b[i][v] + x[v];
        x[v] = a[i][v] * d;
        if constexpr (KIND == SSDQ_GATE_LOG) {
          dg[v] = x[v] * before;
          du[v] = d;
        } else {
          dg[v] = x[v] * cc[i][v] * (before - pu[i][v]);
          du[v] = cc[i][v] * d;
        }
      }
      store_bytes(rdg, base + uint32_t(i) * step, to_pack<T, V>(dg).raw);
      store_bytes(rdu, base + uint32_t(i) * step, to_pack<T, V>(du).raw);
    }
  }
}

// Sets the ticket to 0 and every published word to "not yet".
__global__ void __launch_bounds__(256) gated_clear_kernel(v4u* words, int64_t n, uint32_t* ticket) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i == 0) *ticket = 0;
  for (int64_t k = i; k < n; k += int64_t(gridDim.x) * 256) words[k] = v4u{~0u, ~0u, ~0u, ~0u};
}

// Elementwise over batch * channels: 4 elements per thread (16 bytes of state), whatever the row length.
constexpr int kStep = 4;
template <typename T, int KIND>
__global__ void __launch_bounds__(256) gated_step_kernel(float* __restrict__ state, const T* __restrict__ gate,
                                                         const T* __restrict__ u, T* __restrict__ h, int64_t n) {
  typedef Pack<T, kStep> P;
  typedef typename P::Raw Raw;
  for (int64_t i = (int64_t(blockIdx.x) * 256 + threadIdx.x) * kStep; i < n; i += int64_t(gridDim.x) * 256 * kStep) {
    const bool whole = i + kStep <= n;
    P pg, pu;
    float s[kStep];
    if (whole) {
      pg.raw = *reinterpret_cast<const Raw*>(gate + i);
      pu.raw = *reinterpret_cast<const Raw*>(u + i);
      const v4f v = *reinterpret_cast<const v4f*>(state + i);
#pragma unroll
      for (int e = 0; e < kStep; ++e) s[e] = v[e];
    } else {
      typename P::Elements eg = {}, eu = {};
#pragma unroll
      for (int e = 0; e < kStep; ++e) {
        s[e] = 0.f;
        if (i + e < n) eg.e[e] = gate[i + e], eu.e[e] = u[i + e], s[e] = state[i + e];
      }
      pg.raw = __builtin_bit_cast(Raw, eg);
      pu.raw = __builtin_bit_cast(Raw, eu);
    }
#pragma unroll
    for (int e = 0; e < kStep; ++e) {
      float a, m;
      gate_terms<KIND>(pg[e], a, m);
      s[e] = fmaf(a, s[e], KIND == SSDQ_GATE_LOG ? pu[e] : m * pu[e]);
    }
    const P out = to_pack<T, kStep>(s);
    if (whole) {
      *reinterpret_cast<v4f*>(state + i) = v4f{s[0], s[1], s[2], s[3]};
      *reinterpret_cast<Raw*>(h + i) = out.raw;
    } else {
      const auto e = __builtin_bit_cast(typename P::Elements, out.raw);
#pragma unroll
      for (int k = 0; k < kStep; ++k)
        if (i + k < n) state[i + k] = s[k], h[i + k] = e.e[k];
    }
  }
}

// f(T, KIND) for the runtime dtype and gate kind
template <template <typename, int> class F, typename... A>
hipError_t dispatch(int32_t dtype, int32_t kind, A... args) {
  const bool log = kind == SSDQ_GATE_LOG;
  switch (dtype) {
    case SSDQ_DTYPE_F32: return log ? F<float, SSDQ_GATE_LOG>::run(args...) : F<float, SSDQ_GATE_LOGIT>::run(args...);
    case SSDQ_DTYPE_F16:
      return log ? F<_Float16, SSDQ_GATE_LOG>::run(args...) : F<_Float16, SSDQ_GATE_LOGIT>::run(args...);
    default: return log ? F<__bf16, SSDQ_GATE_LOG>::run(args...) : F<__bf16, SSDQ_GATE_LOGIT>::run(args...);
  }
}

template <typename T, int KIND, int V>
void launch_mode(const GatedArgs& g, const Plan& p, bool back, hipStream_t stream) {
  const dim3 grid(uint32_t(p.tiles) * uint32_t(p.chans)), block(kThreads);
  if (back) {
    if (g.codes) hipLaunchKernelGGL((gated_kernel<T, KIND, V, kBackwardSaved>), grid, block, 0, stream, g, p);
    else hipLaunchKernelGGL((gated_kernel<T, KIND, V, kBackward>), grid, block, 0, stream, g, p);
  } else {
    if (g.codes) hipLaunchKernelGGL((gated_kernel<T, KIND, V, kForwardSave>), grid, block, 0, stream, g, p);
    else hipLaunchKernelGGL((gated_kernel<T, KIND, V, kForward>), grid, block, 0, stream, g, p);
  }
}

template <typename T, int KIND>
struct Scan {
  static hipError_t run(const GatedArgs* g, const Plan* p, bool back, hipStream_t stream) {
    constexpr int kWide = 16 / int(sizeof(T));
    if (g->channels % kWide == 0) launch_mode<T, KIND, kWide>(*g, *p, back, stream);
    else launch_mode<T, KIND, 1>(*g, *p, back, stream);
    return hipGetLastError();
  }
};
template <typename T, int KIND>
struct Step {
  static hipError_t run(float* state, const void* gate, const void* u, void* h, int64_t n, hipStream_t stream) {
    hipLaunchKernelGGL((gated_step_kernel<T, KIND>), dim3(uint32_t(min((n + 256 * kStep - 1) / (256 * kStep), int64_t(1) << 20))),
                       dim3(256), 0, stream, state,
                       static_cast<const T*>(gate), static_cast<const T*>(u), static_cast<T*>(h), n);
    return hipGetLastError();
  }
};

hipError_t launch_scan(const GatedArgs& g, bool back, hipStream_t stream) {
  Plan p = {};
  if (!plan_sizes(g.sequences, g.tokens, g.channels, g.offsets != nullptr, &p)) return hipErrorInvalidValue;
  char* ws = static_cast<char*>(g.workspace);
  p.ticket = reinterpret_cast<uint32_t*>(ws);
  p.maps = reinterpret_cast<uint64_t*>(ws + kTicketBytes);
  if (!p.single) {
    const int64_t words = int64_t(map_bytes(p) / sizeof(v4u));
    const uint32_t blocks = uint32_t(min((words + 255) / 256, int64_t(1024)));
    hipLaunchKernelGGL(gated_clear_kernel, dim3(blocks), dim3(256), 0, stream,
                       reinterpret_cast<v4u*>(ws + kTicketBytes), words, p.ticket);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return dispatch<Scan>(g.dtype, g.gate_kind, &g, &p, back, stream);
}

}  // namespace

size_t gated_workspace_bytes(int32_t sequences, int64_t tokens, int32_t channels, bool packed) {
  Plan p = {};
  if (!plan_sizes(sequences, tokens, channels, packed, &p)) return 0;
  return p.single ? kTicketBytes : kTicketBytes + map_bytes(p);
}

hipError_t launch_gated_scan(const GatedArgs& a, hipStream_t stream) { return launch_scan(a, false, stream); }
hipError_t launch_gated_backward(const GatedArgs& a, hipStream_t stream) { return launch_scan(a, true, stream); }
hipError_t launch_gated_step(int32_t dtype, int32_t gate_kind, float* state, const void* gate, const void* u, void* h,
                             int64_t n, hipStream_t stream) {
  return dispatch<Step>(dtype, gate_kind, state, gate, u, h, n, stream);
}

}  // namespace ssdq
