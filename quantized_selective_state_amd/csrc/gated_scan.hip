// Gated linear recurrence h_t = a_t h_{t-1} + b_t with a gate per channel, its gradient and its
// single-token step (Ternary Mamba, Section 1, states the recurrence).
//
// The maps h -> A h + H compose associatively, (A2, H2) o (A1, H1) = (A2 A1, A2 H1 + H2), so a
// sequence is cut into tiles of 256 (or 128) tokens x 64 channels.  A block of four waves holds one
// tile in registers, as it was loaded: a thread has 16 bytes (8 or 4 neighbouring channels) of 8 or 4
// consecutive tokens.  It composes its tokens' maps, the maps are scanned over the threads of a wave and
// the four waves, the tile's map is published, the state entering the tile is joined from the maps of the
// tiles before it, and each thread runs its tokens once more from its entering state and stores.  Every
// input is read from memory once and every output written once.
//
// The gradient's recurrence k_t = a_t (dh_t + k_{t+1}) is the same scan from a sequence's end with the
// maps (a_t, a_t dh_t), so both directions share the code below.
//
// HBM-bound: under one operation per byte.  A training step of 8 x 4096 x 8192 bf16 (forward with its 8-bit
// checkpoint, backward from it) runs at 5.5 TB/s, a copy of 1 GiB at 5.1.  What that took, beside the single
// pass: enough bytes in flight (64 KB per block and four blocks per CU, hence raw inputs in the registers and the
// gates formed in both passes; persistent blocks with prefetched tiles had half of that and took twice as long),
// channels mapped to XCDs in runs, and non-temporal accesses for large calls.  Gates from logits cost a reciprocal
// more per element (4 x 2048 x 4096 bf16 forward: 52 us a call, from logs in tiles of the same size 50).
#include <algorithm>

#include "gated_types.h"

namespace ssdq {
namespace {

constexpr int kBlock = SSDQ_CHECKPOINT_BLOCK;   // channels of a tile, and of a checkpoint's scale
constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;

constexpr int kForward = 0, kForwardSave = 1;      // with the checkpoint of h written beside h
constexpr int kBackward = 2, kBackwardSaved = 3;   // from the saved h, from its checkpoint
constexpr bool is_back(int mode) { return mode >= kBackward; }

// Tokens of a tile.  A thread holds rows * 64 / 256 elements of each tensor, and no more of them than leaves four blocks
// per CU forward (three in ragged rows with a checkpoint) and three or four backward (two: fp32 logit gates with the
// saved h, and most 16-bit log gates where a block walks two tiles).  256 tokens of a log gate in 16 bits (calls: forward
// 4 x 2048 x 4096 bf16 48 us, 50 with 128; 16384 x 5120 fp16 99 and 109); 128 where a logit's sigmoids are kept too
// (backward 12345 x 2008 fp16 80 us, 92 with 256; 8192 x 4096 fp32 151 and 174) and for 4 bytes (log gates come out
// even there: backward 8192 x 4096 123 and 122 us, 40 packed sequences of 9000 x 2048 74 and 77, 8192 x 1001 53 and 49).
constexpr int tile_rows(int size, int kind) { return size == 4 || kind == SSDQ_GATE_LOGIT ? 128 : 256; }
constexpr int kFewestRows = 128;   // the workspace is sized for any of them

// What a block does: one tile; or, in instances of their own (for the registers), a sequence of several tiles, or also
// short sequences.  Neighbouring sequences that fit in a wave (a quarter of a tile's tokens) together, each in runs of
// tokens of its own, then share it, and a block has four such waves: the same sums in the same order as in a block
// alone.  (256 sequences of 8 tokens x 4096 bf16: 17 us against 71 with a block each.)
constexpr int kTile = 0, kWalk = 1, kShort = 2;
constexpr int runs_of(int size) { return 16 / size; }   // runs of tokens side by side in a wave

// Tiles of a sequence are joined in groups: a tile reads the maps of the tiles of its group before
// it, and of the group before that only the last tile's, which publishes the state it ended with as
// the map (0, state) once it knows that; so does a sequence's first tile.  This fixes the order of every
// product and sum (the same bits on every run) and bounds what a tile reads (16 maps) whatever the length.
constexpr int kGroup = 16;
constexpr int kPeek = 4;   // maps that are read at a time
constexpr int kManyBlocks = 2048;   // twice as many as run at once

// Workspace of chained tiles: a ticket counter per 64 channels, each on a line of its own; for packed sequences
// the table of tiles and the list of waves of short sequences; and the tiles' maps (A, H), in words that are all ones
// until published.  A published word is never all ones: A = NaN is stored with one fixed image.
constexpr size_t kTicketBytes = 128;
constexpr uint64_t kNoMap = ~uint64_t(0);
constexpr int kMostPolls = 1 << 24;   // seconds, far beyond any wait; the state would be NaN if it were ever reached

constexpr int32_t kNoTile = -1, kShared = -2;
struct Tile {
  int32_t seq;       // or kNoTile, or kShared: waves of short sequences, number `chunk` and the next three, of `chunks`
  int32_t chunk;     // tiles of the sequence before this one, in scan order
  int32_t chunks;    // tiles of the sequence
  int32_t base;      // number of the sequence's first tile
  int32_t first;     // the sequence's first row
  int32_t len;       // and its rows
};

struct Plan {
  int32_t tiles;        // most tiles of 64 channels
  int32_t chans;        // blocks of 64 channels
  int32_t per_sequence; // dense: tiles of a sequence (0: packed)
  bool chained;         // some sequence may have more than one tile, or short ones share blocks by the table
  bool sharing;         // short sequences share blocks
  int32_t per_wave;     // one length that fits in a wave: sequences to a wave (else 0)
  bool load_nt, store_nt;   // non-temporal accesses (choose_streams)
  uint32_t* tickets;
  Tile* table;          // packed and chained: the tiles
  uint32_t* shorts;     // and the waves of short sequences: the first one, and how many (2^k) in the top bits
  uint64_t* maps;       // (tiles, chans * 64)
};

int64_t tiles_of(int64_t len, int rows) { return len <= rows ? 1 : (len + rows - 1) / rows; }

// Sizes of a call for tiles of `rows` tokens; false where a launch cannot hold them.
bool plan_sizes(int32_t sequences, int64_t tokens, int32_t channels, bool packed, int rows, int runs, Plan* p) {
  if (channels > (1 << 20)) return false;   // a tile's byte offsets stay below 2^31
  p->chans = (channels + kBlock - 1) / kBlock;
  p->per_sequence = packed ? 0 : int32_t(tiles_of(tokens / sequences, rows));
  p->chained = packed ? tokens > rows : p->per_sequence > 1;
  int64_t tiles = !packed ? int64_t(p->per_sequence) * sequences
                  : p->chained ? tokens / rows + sequences : sequences;
  if (tiles * p->chans >= (int64_t(1) << 24)) return false;   // a grid holds fewer than 2^32 threads
  const int64_t fits = rows / kWaves;
  if (packed) {
    // The table of tiles is worth its launch where a block per sequence would be more blocks than run at once (200 tokens
    // x 4096 bf16, a call with the table against one without: 60 sequences 15.9 and 17.9 us, 40 sequences 15.9 and
    // 13.4, 20 sequences 15.6 and 12.9), and sharing where sequences are shorter than a tile on average (200 sequences,
    // 8192 tokens x 4096: 63 us against 86; 150 sequences, 2000 tokens, training step: 59 against 144).
    p->chained = p->chained || int64_t(sequences) * p->chans > kManyBlocks;
    p->sharing = p->chained && tokens / rows < sequences;
    const int64_t most = std::min(int64_t(sequences), tokens / (fits + 1));   // sequences that do not fit in a wave
    if (p->sharing) tiles = tokens / rows + most + (sequences - most + kWaves - 1) / kWaves;
    else if (p->chained) tiles = tokens / rows + sequences;
  } else if (tokens / sequences <= fits) {
    p->sharing = true;
    const int64_t len = tokens / sequences, run = fits / runs;
    p->per_wave = int32_t(runs / std::max(int64_t(1), (len + run - 1) / run));
    tiles = (int64_t(sequences) + p->per_wave * kWaves - 1) / (p->per_wave * kWaves);
  }
  p->tiles = int32_t(tiles);
  return true;
}
size_t round_up(size_t n) { return (n + 255) & ~size_t(255); }
size_t ticket_bytes(const Plan& p) { return round_up(size_t(p.chans) * kTicketBytes); }
size_t table_bytes(const Plan& p) { return p.per_sequence ? 0 : round_up(size_t(p.tiles) * sizeof(Tile)); }
size_t short_bytes(int32_t sequences, const Plan& p) {
  return p.per_sequence ? 0 : round_up(size_t(sequences) * sizeof(int32_t));
}
size_t map_bytes(const Plan& p) { return size_t(p.tiles) * p.chans * kBlock * sizeof(uint64_t); }

// Buffer accesses: out-of-range reads give zeros, out-of-range writes are dropped.  NT: non-temporal.
constexpr int kNt = 2;
template <bool NT = false>
__device__ __forceinline__ void load_bytes(Rsrc r, uint32_t off, v4u& v) {
  v = __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, NT ? kNt : 0);
}
template <bool NT = false>
__device__ __forceinline__ void load_bytes(Rsrc r, uint32_t off, v2u& v) {
  v = __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, NT ? kNt : 0);
}
template <bool NT = false>
__device__ __forceinline__ void load_bytes(Rsrc r, uint32_t off, uint32_t& v) {
  v = __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, NT ? kNt : 0);
}
template <bool NT = false>
__device__ __forceinline__ void store_bytes(Rsrc r, uint32_t off, v4u v) {
  __builtin_amdgcn_raw_buffer_store_b128(v, r, off, 0, NT ? kNt : 0);
}
template <bool NT = false>
__device__ __forceinline__ void store_bytes(Rsrc r, uint32_t off, v2u v) {
  __builtin_amdgcn_raw_buffer_store_b64(v, r, off, 0, NT ? kNt : 0);
}
template <bool NT = false>
__device__ __forceinline__ void store_bytes(Rsrc r, uint32_t off, uint32_t v) {
  __builtin_amdgcn_raw_buffer_store_b32(v, r, off, 0, NT ? kNt : 0);
}

// The rows of a tile of one tensor, V elements at a time, through buffer accesses.  RAGGED rows (whose length
// is no multiple of V) start at any multiple of the element's size, and in the last block of channels (`ends`) one
// lane of a row has fewer than V elements, `tail`.  A load takes the aligned words that hold the elements (one
// more than they fill) and shifts them when all tensors' loads are under way; where rows end, word by
// word.  A store goes to the unaligned address as a plain access, that of a tail in pieces of 8, 4, 2 and 1 bytes.
template <typename T, int V, int R, bool RAGGED>
struct Rows {
  typedef Pack<T, V> P;
  typedef typename P::Raw Raw;
  static constexpr int S = sizeof(T), kBytes = S * V, kWords = kBytes / 4;
  static constexpr bool kShifted = RAGGED && S < 4;   // rows of 4-byte elements start at whole words
  struct __attribute__((packed, aligned(S))) Loose { Raw v; };
  template <typename W>
  struct __attribute__((packed, aligned(S))) Piece { W v; };
  struct Words { uint32_t w[kWords]; };
  struct Staged { Words x; uint32_t behind; };
  Rsrc rsrc;
  char* base;
  uint32_t bytes, shift;   // shift: of the first row's address from a whole word
  int tail;
  bool odd, ends, nt;
  __device__ __forceinline__ Rows(const T* p, uint32_t n, int32_t channels, bool last, bool stream)
      : base(reinterpret_cast<char*>(const_cast<T*>(p))), bytes(n), shift(0), tail(0), odd(false), ends(false),
        nt(stream) {
    if constexpr (RAGGED) {
      odd = channels * S % 4 != 0;
      if constexpr (kShifted) shift = uint32_t(reinterpret_cast<uintptr_t>(p)) & 3u;
      tail = channels % V;
      ends = last;
    }
    // the last row's last word may end past the row
    rsrc = make_rsrc(base - shift, kShifted && n ? n + shift + 3u : n);
  }
  // f(piece of W, its byte offset among the tail's elements) for every piece of the tail
  template <typename F>
  __device__ __forceinline__ void pieces(F f) const {
    int at = 0;
    if constexpr (kBytes > 8)
      if (tail * S & 8) f(uint64_t{}, at), at += 8;
    if constexpr (kBytes > 4 && S <= 4)
      if (tail * S & 4) f(uint32_t{}, at), at += 4;
    if constexpr (S <= 2)
      if (tail * S & 2) f(u16{}, at), at += 2;
    if constexpr (S == 1)
      if (tail & 1) f(uint8_t{}, at);
  }
  // off(i): byte offset of the i-th of R packs, out of range where there is none; count: the lane's elements
  template <typename F>
  __device__ __forceinline__ void stage(Staged (&v)[R], F off, int count) const {
    // Every word read holds at least one byte of the row: V elements have another one of the row behind them (its
    // tail), and at a row's end no word is read that starts past it.
    const auto word = [&](int i) { return off(i) < bytes ? (off(i) + shift) & ~3u : kOutOfRange; };
    if (RAGGED && ends) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const uint32_t end = off(i) + shift + uint32_t(max(min(count, V), 0) * S);
#pragma unroll
        for (int k = 0; k <= kWords; ++k) {
          const uint32_t at = word(i) + 4u * uint32_t(k);
          uint32_t got = 0;
          if (k < kWords || kShifted) load_bytes(rsrc, at < end ? at : kOutOfRange, got);
          if (k < kWords) v[i].x.w[k] = got;
          else v[i].behind = got;
        }
      }
    } else if (!RAGGED && nt) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        Raw raw;
        load_bytes<true>(rsrc, off(i), raw);
        v[i].x = __builtin_bit_cast(Words, raw);
      }
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        Raw raw;
        load_bytes(rsrc, RAGGED ? word(i) : off(i), raw);
        v[i].x = __builtin_bit_cast(Words, raw);
        v[i].behind = 0;
        if constexpr (kShifted) load_bytes(rsrc, word(i) + uint32_t(kBytes), v[i].behind);
      }
    }
  }
  template <typename F>
  __device__ __forceinline__ void finish(P (&v)[R], const Staged (&from)[R], F off) const {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      Words x = from[i].x;
      if constexpr (kShifted) {
        const uint32_t by = 8u * ((off(i) + shift) & 3u);
#pragma unroll
        for (int k = 0; k < kWords; ++k)
          x.w[k] = __builtin_amdgcn_alignbit(k + 1 < kWords ? from[i].x.w[k + 1] : from[i].behind, from[i].x.w[k], by);
      }
      v[i].raw = __builtin_bit_cast(Raw, x);
    }
  }
  __device__ __forceinline__ void store(uint32_t off, int count, P v) const {
    // (where rows are whole words, a buffer access would do; one that is unaligned is left to the compiler)
    if (RAGGED && odd) {
      if (off < bytes && count >= V) reinterpret_cast<Loose*>(base + off)->v = v.raw;
    } else if (!RAGGED && nt) {
      store_bytes<true>(rsrc, off, v.raw);
    } else {
      store_bytes(RAGGED ? make_rsrc(base, bytes) : rsrc, RAGGED && count < V ? kOutOfRange : off, v.raw);
    }
    if (RAGGED && ends) {
      if (count > 0 && count < V && off < bytes) {
        const Words x = __builtin_bit_cast(Words, v.raw);
        pieces([&](auto piece, int o) {
          typedef decltype(piece) W;
          uint64_t word = 0;
          if constexpr (sizeof(W) == 8) {
            word = uint64_t(x.w[0]) | uint64_t(x.w[1]) << 32;
          } else {
#pragma unroll
            for (int k = 0; k < kWords; ++k)
              if (o / 4 == k) word = x.w[k] >> (8 * (o % 4));
          }
          reinterpret_cast<Piece<W>*>(base + off + o)->v = W(word);
        });
      }
    }
  }
};

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


// Makes the second pass form a and b again from what is kept, instead of keeping those from the first.
__device__ __forceinline__ void opaque(v4u& v) { asm volatile("" : "+v"(v)); }
__device__ __forceinline__ void opaque(float& v) { asm volatile("" : "+v"(v)); }

// What the waves of a block exchange.
struct Shared {
  float A[kWaves][kBlock], H[kWaves][kBlock];   // the waves' maps
  float in[kBlock];                             // the state entering the tile
  int32_t ticket;
};

// One tile.  carry: where a block walks its sequence, the state after the tile before, and then after this one (a lane
// of the first wave per channel).  TOGETHER: a wave has whole sequences of its own, t.chunks of them (or none) from t.seq,
// in the rows t.first and t.len.
template <typename T, int KIND, int MODE, bool RAGGED, bool TOGETHER>
__device__ __forceinline__ void run_tile(const GatedArgs& g, const Plan& p, const Tile& t, int32_t blk, Shared& sh,
                                         float& carry) {
  constexpr bool kBack = is_back(MODE);
  constexpr int ROWS = tile_rows(sizeof(T), KIND);
  constexpr int V = 16 / int(sizeof(T)); // channels of a thread
  constexpr int LPR = kBlock / V;        // lanes of a row
  constexpr int kRuns = kWave / LPR;     // runs of tokens in a wave
  constexpr int R = ROWS / (kWaves * kRuns);   // tokens of a run
  static_assert(R >= 1 && R * kWaves * kRuns == ROWS, "a block holds one tile");
  typedef Pack<T, V> P;
  typedef Rows<T, V, R, RAGGED> Rw;
  typedef Rows<int8_t, V, R, RAGGED> Rc;

  const int tid = int(threadIdx.x), lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  const int32_t nrows = min(ROWS, t.len - t.chunk * ROWS);
  // rows of the tile: the scan runs from the first to the last, or from the last to the first
  const int64_t row0 = kBack ? int64_t(t.first) + t.len - t.chunk * ROWS - nrows : int64_t(t.first) + t.chunk * ROWS;
  const int64_t start = row0 * g.channels;

  const int group = lane / LPR, col = (lane % LPR) * V;
  const int c = blk * kBlock + col, count = min(V, g.channels - c);
  const bool in = c < g.channels, ends = blk == p.chans - 1;
  const uint32_t width = uint32_t(g.channels) * uint32_t(sizeof(T)), crow = uint32_t(g.channels);
  const uint32_t srow = 4u * uint32_t(p.chans);
  const int slot = TOGETHER ? 0 : wave;
  // the lane's run: its sequence, which of that one's runs in this wave it is, the scan position of its first token, how
  // many tokens come from there on, and the row of the first one in the tile
  int32_t seq = t.seq;
  int rank = group, run = (slot * kRuns + group) * R, left = nrows - run, row = kBack ? left - 1 : run;
  bool closes = group == min(kRuns - 1, max(nrows - slot * kRuns * R - 1, 0) / R);   // the last with tokens
  if constexpr (TOGETHER) {
    int32_t lo = 0, hi = 0;
    if (lane < t.chunks) {
      if (p.per_wave) lo = (t.seq + lane) * int32_t(g.tokens / g.sequences), hi = lo + int32_t(g.tokens / g.sequences);
      else sequence_rows(g, t.seq + lane, lo, hi);
    }
    int at = 0, mine = 0, before = 0, of = 0, first = 0, len = 0;   // at: runs given to the sequences so far
    for (int j = 0; j < t.chunks; ++j) {
      const int f = __builtin_amdgcn_readlane(lo, j), n = __builtin_amdgcn_readlane(hi, j) - f;
      const int runs = max(1, (n + R - 1) / R);
      if (group >= at) mine = j, before = at, of = runs, first = f, len = n;
      at += runs;
    }
    rank = group - before;
    run = rank * R;
    // (sequences that overlap or leave the tile's rows, of offsets out of order, are left out)
    const bool is = t.chunks > 0 && rank < of && first >= t.first && first - t.first <= nrows - len;
    seq = is ? t.seq + mine : -1;
    left = is ? len - run : 0;
    row = first - t.first + (kBack ? left - 1 : run);
    closes = is && rank == of - 1;
  }
  const bool busy = slot * kRuns * R < nrows;   // a wave without rows holds the identity and stores nothing
  // byte offset of token i of the run in rows of `w` bytes, `at` into the row; past the tile's rows it is out of
  // range (below row 0 it wraps to above 2^31), and so it is for a lane past the channels
  const auto offset = [&](int i, uint32_t w, uint32_t at) {
    if constexpr (TOGETHER) return in && i < left ? uint32_t(kBack ? row - i : row + i) * w + at : kOutOfRange;
    return in ? uint32_t(kBack ? nrows - 1 - run - i : run + i) * w + at : kOutOfRange;
  };
  const auto at_t = [&](int i) { return offset(i, width, uint32_t(c) * uint32_t(sizeof(T))); };
  const auto at_c = [&](int i) { return offset(i, crow, uint32_t(c)); };
  const auto at_s = [&](int i) { return offset(i, srow, 4u * uint32_t(blk)); };
  const auto rows_of = [&](const void* x, bool nt) {
    return Rw(static_cast<const T*>(x) + start, uint32_t(nrows) * width, g.channels, ends, nt);
  };

  const Rw rg = rows_of(g.gate, p.load_nt), rs = rows_of(kBack ? g.dh : g.u, p.load_nt);
  typename Rw::Staged vg[R], vs[R], vh[R], vu[R];
  typename Rc::Staged vc[R];
  if (busy) {
    rg.stage(vg, at_t, count);
    rs.stage(vs, at_t, count);
  }
  // The states that the tokens start from are those of the row before; the sequence's first token starts from
  // h0, and its row is out of range.
  const int first_at = kBack && row0 == t.first ? left - 1 : -1;   // that token's place in the run
  const auto at_h = [&](int i) { return i == first_at ? kOutOfRange : at_t(i); };
  const auto at_hc = [&](int i) { return i == first_at ? kOutOfRange : at_c(i); };
  const T* const hbase = MODE == kBackward ? static_cast<const T*>(g.h) + (start - g.channels) : nullptr;
  const int8_t* const cbase = MODE == kBackwardSaved ? g.codes + (start - g.channels) : nullptr;
  const Rw rh(hbase, uint32_t(nrows) * width, g.channels, ends, p.load_nt), ru = rows_of(g.u, p.load_nt);
  const Rc rc(cbase, uint32_t(nrows) * crow, g.channels, ends, false);
  float sc[R];
  if (busy) {
    if constexpr (MODE == kBackward) rh.stage(vh, at_h, count);
    if constexpr (MODE == kBackwardSaved) {
      rc.stage(vc, at_hc, count);
      const Rsrc rscale = make_rsrc(g.scale + (row0 - 1) * p.chans, uint32_t(nrows) * srow);
#pragma unroll
      for (int i = 0; i < R; ++i) sc[i] = buf_loadf(rscale, i == first_at ? kOutOfRange : at_s(i));
    }
    if constexpr (kBack && KIND == SSDQ_GATE_LOGIT) ru.stage(vu, at_t, count);
  }
  P pg[R], ps[R], ph[R], pu[R];
  Pack<int8_t, V> pc[R];
  if (busy) {
    rg.finish(pg, vg, at_t);
    rs.finish(ps, vs, at_t);
    if constexpr (MODE == kBackward) rh.finish(ph, vh, at_h);
    if constexpr (MODE == kBackwardSaved) rc.finish(pc, vc, at_hc);
    if constexpr (kBack && KIND == SSDQ_GATE_LOGIT) ru.finish(pu, vu, at_t);
  }

  // A row past the tile has gate and input 0: the identity for a log gate.  For a logit it is +infinity.
  if constexpr (KIND == SSDQ_GATE_LOGIT) {
    if (TOGETHER || nrows < ROWS) {
      float inf[V];
#pragma unroll
      for (int v = 0; v < V; ++v) inf[v] = __builtin_inff();
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (i >= left) pg[i] = to_pack<T, V>(inf);
    }
  }
  // A token's a, what it adds (backward: dh) and what multiplies its input; again: in the second pass.  A log
  // gate's exponential is formed twice, a logit's sigmoids are kept as one number.
  float pair[R][V];
  const auto token = [&](int i, int v, bool again, float& a, float& b, float& m) {
    if constexpr (KIND == SSDQ_GATE_LOG) {
      gate_terms<KIND, sizeof(T) == 4>(pg[i][v], a, m);
      b = ps[i][v];
    } else {
      if (!again) pair[i][v] = logit_pair<sizeof(T) == 4>(pg[i][v]);
      split_pair(pair[i][v], a, m);
      b = kBack ? ps[i][v] : m * ps[i][v];
    }
  };
  float A[V], H[V];
#pragma unroll
  for (int v = 0; v < V; ++v) A[v] = 1.f, H[v] = 0.f;
  if (busy) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float a, b, m;
        token(i, v, false, a, b, m);
        A[v] *= a;
        H[v] = kBack ? a * (b + H[v]) : fmaf(a, H[v], b);
      }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if constexpr (KIND == SSDQ_GATE_LOG) {
        opaque(pg[i].raw);
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v) opaque(pair[i][v]);
      }
      opaque(ps[i].raw);
    }
    // inclusive scan of the runs' maps within the wave
#pragma unroll
    for (int o = 1; o < kRuns; o <<= 1) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float pA = __shfl_up(A[v], o * LPR, 64), pH = __shfl_up(H[v], o * LPR, 64);
        if (rank >= o) {
          H[v] = fmaf(A[v], pH, H[v]);
          A[v] *= pA;
        }
      }
    }
  }
  const float* const init = kBack ? g.dh_final : g.h0;
  float* const out = kBack ? g.dh0 : g.h_final;
  float x[V];   // the state that enters the run; together: first that which the sequence starts from
  if constexpr (TOGETHER) {
    const int64_t at = int64_t(seq) * g.channels + c;
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = init && seq >= 0 && v < count ? init[at + v] : 0.f;
    if (out && closes) {
      // (the whole wave has read the first states, which these may overwrite)
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (v < count) out[at + v] = run + left ? fmaf(A[v], x[v], H[v]) : x[v];
    }
  } else if (closes) {
#pragma unroll
    for (int v = 0; v < V; ++v) sh.A[wave][col + v] = A[v], sh.H[wave][col + v] = H[v];
  }
  // each run's exclusive map
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const float pA = __shfl_up(A[v], LPR, 64), pH = __shfl_up(H[v], LPR, 64);
    A[v] = rank ? pA : 1.f;
    H[v] = rank ? pH : 0.f;
  }
  __syncthreads();

  if (wave == 0 && !TOGETHER) {
    // a lane per channel: the tile's map, and the state entering the tile
    const int64_t cpad = int64_t(p.chans) * kBlock, ch = int64_t(blk) * kBlock + lane;
    const bool some = ch < g.channels;
    const int64_t at = int64_t(t.seq) * g.channels + ch;
    float tA = 1.f, tH = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      tH = fmaf(sh.A[w][lane], tH, sh.H[w][lane]);
      tA *= sh.A[w][lane];
    }
    const bool last = t.chunk == t.chunks - 1, ends_group = t.chunk % kGroup == kGroup - 1;
    uint64_t* maps = p.maps + int64_t(t.base) * cpad + ch;
    float first_state = 0.f;
    if (t.chunk == 0) {
      // only this tile reads the initial state (which the final one may overwrite)
      first_state = some && init ? init[at] : 0.f;
    } else if (!p.chained) {
      first_state = carry;
    } else {
      if (!last && !ends_group) publish(maps + int64_t(t.chunk) * cpad, map_word(tA, tH));
      const int from = max(t.chunk / kGroup * kGroup - 1, 0), n = t.chunk - from;
#pragma unroll 1
      for (int j0 = 0; j0 < n; j0 += kPeek) {
        uint64_t got[kPeek];
        for (int polls = 0;; ++polls) {
          bool all = true;
#pragma unroll
          for (int j = 0; j < kPeek; ++j) {
            got[j] = peek(maps + int64_t(from + min(j0 + j, n - 1)) * cpad);
            all = all && got[j] != kNoMap;
          }
          if (__all(all) || polls == kMostPolls) break;
          __builtin_amdgcn_s_sleep(1);
        }
#pragma unroll
        for (int j = 0; j < kPeek; ++j)
          if (j0 + j < n)
            first_state = fmaf(__uint_as_float(uint32_t(got[j])), first_state, __uint_as_float(uint32_t(got[j] >> 32)));
      }
    }
    sh.in[lane] = first_state;
    carry = fmaf(tA, first_state, tH);
    if (p.chained && !last && (t.chunk == 0 || ends_group))
      publish(maps + int64_t(t.chunk) * cpad, map_word(0.f, carry));
    if (last && out && some) out[at] = t.len ? carry : first_state;
  }
  __syncthreads();
  if constexpr (!TOGETHER) {
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = sh.in[col + v];
  }
  if (!busy) return;   // (the block goes on behind the tile)

  // the state entering each run: the tile's, then the waves before, then the runs before
  for (int w = 0; w < slot; ++w) {
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = fmaf(sh.A[w][col + v], x[v], sh.H[w][col + v]);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) x[v] = fmaf(A[v], x[v], H[v]);

  if constexpr (!kBack) {
    const Rw out_rows = rows_of(g.h, p.store_nt);
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float a, b, m;
        token(i, v, true, a, b, m);
        x[v] = fmaf(a, x[v], b);
      }
      const P out = to_pack<T, V>(x);
      out_rows.store(at_t(i), count, out);
      if constexpr (MODE == kForwardSave) {
        const float scale = checkpoint_scale(row_umax<LPR>(largest<T, V>(out, RAGGED ? count : in ? V : 0)));
        const Rc out_codes(g.codes + start, uint32_t(nrows) * crow, g.channels, ends, false);
        const Rsrc out_scale = make_rsrc(g.scale + row0 * p.chans, uint32_t(nrows) * srow);
        out_codes.store(at_c(i), count, Pack<int8_t, V>{codes_of<V>(out, scale)});
        store_bytes(out_scale, col == 0 ? at_s(i) : kOutOfRange, __float_as_uint(scale));
      }
    }
  } else {
    const Rw rdg = rows_of(g.dgate, p.store_nt), rdu = rows_of(g.du, p.store_nt);
    float h0[V];
#pragma unroll
    for (int v = 0; v < V; ++v) h0[v] = 0.f;
    if (g.h0 && first_at >= 0 && first_at < R) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (v < count) h0[v] = g.h0[int64_t(seq) * g.channels + c + v];
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float dg[V], du[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float a, b, m, before;
        token(i, v, true, a, b, m);
        if constexpr (MODE == kBackward) before = ph[i][v];
        else before = pc[i][v] * sc[i];
        if (i == first_at) before = h0[v];
        const float d = b + x[v];
        x[v] = a * d;
        if constexpr (KIND == SSDQ_GATE_LOG) {
          dg[v] = x[v] * before;
          du[v] = d;
        } else {
          dg[v] = x[v] * m * (before - pu[i][v]);
          du[v] = m * d;
        }
      }
      rdg.store(at_t(i), count, to_pack<T, V>(dg));
      rdu.store(at_t(i), count, to_pack<T, V>(du));
    }
  }
}

template <typename T, int KIND, int MODE, bool RAGGED, int WORK>
__global__ void __launch_bounds__(kThreads) gated_kernel(GatedArgs g, Plan p) {
  __shared__ Shared sh;
  // A block's channels go by its number, so that neighbouring channels of the same rows run on one XCD: its
  // blocks then use all channels of its L2.  (With the 8 XCDs' blocks interleaved, each XCD met only the
  // lines of one residue mod 1 KB: forward 16384 x 5120 fp16 108 us against 99, training step 8 x 4096 x 8192 bf16 868
  // against 787, packed 12345 x 2008 91 against 80; of the cases measured only backward 8192 x 4096 fp32 had it the other
  // way, 120 against 124.)
  const int32_t blk = xcd_remap(int32_t(blockIdx.x % uint32_t(p.chans)), p.chans);
  int32_t index = int32_t(blockIdx.x / uint32_t(p.chans));
  if (p.chained) {
    // Tiles are taken by tickets, in the order in which blocks start, so that a tile's predecessors (lower
    // tickets of the same channels) are held by blocks that run already and publish before they wait for anything
    // but lower tickets: every wait ends.  One counter for all channels would serialize the starts (3.4 ns each).
    if (threadIdx.x == 0)
      sh.ticket = int32_t(__hip_atomic_fetch_add(p.tickets + size_t(blk) * (kTicketBytes / sizeof(uint32_t)), 1u,
                                               __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
    __syncthreads();
    index = __builtin_amdgcn_readfirstlane(sh.ticket);
  }
  Tile t;
  bool together = false;
  const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
  if (WORK == kShort && p.per_wave) {
    const int64_t first = (int64_t(index) * kWaves + wave) * p.per_wave;
    t = Tile{int32_t(min(first, int64_t(g.sequences))), 0, 0, 0, 0, 0};
    t.chunks = min(p.per_wave, g.sequences - t.seq);
    t.first = t.seq * int32_t(g.tokens / g.sequences);
    t.len = t.chunks * int32_t(g.tokens / g.sequences);
    together = true;
  } else if (p.per_sequence) {
    // dense: the first tiles of all sequences, then their second ones, ...
    t.chunk = index / g.sequences;
    t.seq = index - t.chunk * g.sequences;
    t.chunks = p.per_sequence;
    t.base = t.seq * p.per_sequence;
    t.len = int32_t(g.tokens / g.sequences);
    t.first = t.seq * t.len;
  } else {
    t = p.chained ? p.table[index] : Tile{index, 0, 1, 0, 0, 0};
    if (t.seq == kNoTile) return;
    together = WORK == kShort && t.seq == kShared;
    if (together) {
      const int32_t k = t.chunk + wave;
      const bool is = k < t.chunks;
      const uint32_t w = is ? p.shorts[k] : 0u;
      t = Tile{int32_t(w & 0xFFFFFFu), 0, 0, 0, 0, 0};
      if (is) {
        t.chunks = min(int32_t(1u << (w >> 24)), g.sequences - t.seq);
        int32_t end, ignored;
        sequence_rows(g, t.seq, t.first, end);
        sequence_rows(g, t.seq + t.chunks - 1, ignored, end);
        t.len = max(end - t.first, 0);
      }
    } else if (!p.chained) {
      int32_t end;
      sequence_rows(g, t.seq, t.first, end);
      t.len = end - t.first;
    }
    together = __builtin_amdgcn_readfirstlane(together);
  }
  // (scalar registers for all that follows from the tile, the buffer descriptors among it)
  t = Tile{__builtin_amdgcn_readfirstlane(t.seq),  __builtin_amdgcn_readfirstlane(t.chunk),
           __builtin_amdgcn_readfirstlane(t.chunks), __builtin_amdgcn_readfirstlane(t.base),
           __builtin_amdgcn_readfirstlane(t.first), __builtin_amdgcn_readfirstlane(t.len)};
  float carry = 0.f;
  if constexpr (WORK == kShort) {
    if (together) return run_tile<T, KIND, MODE, RAGGED, true>(g, p, t, blk, sh, carry);
  }
  run_tile<T, KIND, MODE, RAGGED, false>(g, p, t, blk, sh, carry);
  if constexpr (WORK == kWalk) {
    while (++t.chunk < t.chunks) {
      __syncthreads();   // every wave has read the maps of the tile before
      run_tile<T, KIND, MODE, RAGGED, false>(g, p, t, blk, sh, carry);
    }
  }
}

// Before chained tiles: the tickets to 0, every map to "not yet", and for packed sequences the table of
// tiles, by the last block: those of the sequences that do not fit in a wave, then those of waves of short ones (of 8,
// 4 or 2 sequences whose number starts at a multiple of that, if they fit in a wave together, or of one).
//
// 4 to 6 us, bound by the launch, up to some hundred sequences; the one block that makes the table then takes 4.1 us per
// 1000 sequences (10,000 sequences of 8 tokens x 256 bf16: 43 of the call's 110 us, as a dense call 34 us).
__global__ void __launch_bounds__(256) gated_clear_kernel(GatedArgs g, Plan p, int64_t zeros, int64_t words,
                                                          int rows, int runs) {
  const bool packed = p.per_sequence == 0;
  if (packed && blockIdx.x == gridDim.x - 1) {
    __shared__ Tile seq[256];
    const int tid = int(threadIdx.x), lane = tid & 63, wave = tid >> 6;
    __shared__ int64_t sums[4];
    __shared__ int32_t counts[4];
    int64_t base = 0;   // in 64 bits: overlapping sequences could have any number of tiles
    int32_t shorts = 0;
    for (int s0 = 0; s0 < g.sequences && base < p.tiles; s0 += 256) {
      int32_t lo = 0, hi = 0, n = 0;
      bool fits = false;
      if (s0 + tid < g.sequences) {
        sequence_rows(g, s0 + tid, lo, hi);
        fits = p.sharing && hi - lo <= rows / kWaves;
        n = fits ? 0 : hi - lo <= rows ? 1 : (hi - lo + rows - 1) / rows;
      }
      const int run = rows / kWaves / runs;
      const int one = s0 + tid >= g.sequences ? 0 : fits ? max(1, (hi - lo + run - 1) / run) : runs + 1;
      const int two = one + __shfl_xor(one, 1, 64), four = two + __shfl_xor(two, 2, 64);
      const int log = four + __shfl_xor(four, 4, 64) <= runs ? 3 : four <= runs ? 2 : two <= runs ? 1 : 0;
      fits = fits && tid % (1 << log) == 0;   // the first sequence of a wave
      const uint64_t fitting = __ballot(fits);
      int64_t upto = n;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int64_t v = __shfl_up(upto, o, 64);
        if (lane >= o) upto += v;
      }
      __syncthreads();   // the strip before is in the table
      if (lane == 63) sums[wave] = upto, counts[wave] = __popcll(fitting);
      __syncthreads();
      int64_t total = 0;
      int32_t at = shorts + __popcll(fitting & ((uint64_t(1) << lane) - 1));
      for (int w = 0; w < 4; ++w) {
        if (w < wave) upto += sums[w], at += counts[w];
        total += sums[w];
        shorts += counts[w];
      }
      if (fits) p.shorts[at] = uint32_t(s0 + tid) | uint32_t(log) << 24;
      const int64_t mine = base + upto - n;
      seq[tid] = Tile{s0 + tid, 0, n, int32_t(mine < p.tiles ? mine : p.tiles), lo, hi - lo};
      __syncthreads();
      // tiles past the table's end (of overlapping sequences) are left out
      const int32_t end = int32_t(base + total < p.tiles ? base + total : p.tiles);
      for (int32_t i = int32_t(base) + tid; i < end; i += 256) {
        int k = 0;
        for (int step = 128; step >= 1; step >>= 1)
          if (seq[k + step].base <= i) k += step;   // the last sequence of the strip that starts at i or before
        Tile t = seq[k];
        t.chunk = i - t.base;
        p.table[i] = t;
      }
      base += total;
    }
    for (int64_t i = base + tid; i < p.tiles; i += 256) {
      const int64_t k = (i - base) * kWaves;
      p.table[i] = Tile{k < shorts ? kShared : kNoTile, int32_t(k < shorts ? k : 0), shorts, 0, 0, 0};
    }
    return;
  }
  const int64_t stride = int64_t(gridDim.x - (packed ? 1 : 0)) * 256;
  const int64_t first = int64_t(blockIdx.x) * 256 + threadIdx.x;
  v4u* tickets = reinterpret_cast<v4u*>(p.tickets);
  v4u* maps = reinterpret_cast<v4u*>(p.maps);
  for (int64_t k = first; k < zeros; k += stride) tickets[k] = v4u{0u, 0u, 0u, 0u};
  for (int64_t k = first; k < words; k += stride) maps[k] = v4u{~0u, ~0u, ~0u, ~0u};
}

// The step: elementwise over batch * channels, 4 elements per thread (16 bytes of state), whatever the row length.
// HBM-bound (14 bytes per element of 16 bits): 6.3 us at 256 x 8192 fp16, 4.7 TB/s; the call itself takes 7.8.
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
      gate_terms<KIND, sizeof(T) == 4>(pg[e], a, m);
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

template <typename T, int KIND, bool RAGGED, int WORK>
void launch_mode(const GatedArgs& g, const Plan& p, bool back, hipStream_t stream) {
  const dim3 grid(uint32_t(p.tiles) * uint32_t(p.chans)), block(kThreads);
  if (back) {
    if (g.codes)
      hipLaunchKernelGGL((gated_kernel<T, KIND, kBackwardSaved, RAGGED, WORK>), grid, block, 0, stream, g, p);
    else hipLaunchKernelGGL((gated_kernel<T, KIND, kBackward, RAGGED, WORK>), grid, block, 0, stream, g, p);
  } else {
    if (g.codes) hipLaunchKernelGGL((gated_kernel<T, KIND, kForwardSave, RAGGED, WORK>), grid, block, 0, stream, g, p);
    else hipLaunchKernelGGL((gated_kernel<T, KIND, kForward, RAGGED, WORK>), grid, block, 0, stream, g, p);
  }
}

// Non-temporal accesses, for rows of whole 128-byte lines (lines that two blocks share are worth keeping: training
// step 32768 x 8200 bf16 1254 us against 1585).  Loads, once a call touches more than the 256 MiB of the Infinity Cache,
// since what a call reads is then gone before anything reads it again (forward 16384 x 5120 fp16 108 -> 99 us, backward
// 8192 x 4096 fp32 143 -> 123; below, 2 x 2048 x 4096 bf16, 23.6 us against 28.2 with them); stores, once the outputs
// alone do (training step 32768 x 8192 bf16 902 -> 787 us with both; a smaller output stays for what reads it: backward
// fp32 above 123 against 135 us).  A logit gate's gradient too, which reads four tensors: 4 x 4096 x 8192 bf16 327 -> 307
// us from h and 306 -> 288 from a checkpoint, fp32 from h 600 -> 541.
void choose_streams(const GatedArgs& g, int kind, bool back, int size, Plan* p) {
  constexpr int64_t kCache = int64_t(256) << 20;
  const int64_t tensor = g.tokens * g.channels * size, outputs = (back ? 2 : 1) * tensor;
  const int64_t saved = !back ? 0 : g.codes ? tensor / size : tensor;
  const int64_t inputs = (back && kind == SSDQ_GATE_LOGIT ? 3 : 2) * tensor + saved;
  const bool lines = int64_t(g.channels) * size % 128 == 0;
  p->load_nt = lines && inputs + outputs > kCache;
  p->store_nt = lines && outputs > kCache;
}

template <typename T, int KIND>
struct Scan {
  static hipError_t run(const GatedArgs* g, bool back, hipStream_t stream) {
    const int rows = tile_rows(sizeof(T), KIND);
    Plan p = {};
    if (!plan_sizes(g->sequences, g->tokens, g->channels, g->offsets != nullptr, rows, runs_of(sizeof(T)), &p))
      return hipErrorInvalidValue;
    // Two tiles: one block for both, and no maps to clear.  Calls of 1, 8, 64 sequences walked, and chained through maps:
    // 512 tokens x 4096 bf16 log, forward 13.0, 22.5, 141 and 15.6, 23.1, 144 us, training step 36, 70, 425 and 41, 76,
    // 423 (4 sequences are the one loss: 45.5 and 40.8); 256 tokens, logit, training step 35, 46.5, 260 and 39, 47.5, 265;
    // fp32 log, backward 15.7, 38, 258 and 18, 43, 269.  One sequence of three tiles would take 15 walked, 14 chained.
    const bool walk = p.per_sequence == 2;
    if (walk) p.chained = false, p.tiles = g->sequences;
    if (p.chained) {
      char* ws = static_cast<char*>(g->workspace);
      p.tickets = reinterpret_cast<uint32_t*>(ws);
      p.table = reinterpret_cast<Tile*>(ws + ticket_bytes(p));
      p.shorts = reinterpret_cast<uint32_t*>(ws + ticket_bytes(p) + table_bytes(p));
      p.maps = reinterpret_cast<uint64_t*>(ws + ticket_bytes(p) + table_bytes(p) + short_bytes(g->sequences, p));
      const int64_t zeros = int64_t(ticket_bytes(p) / sizeof(v4u)), words = int64_t(map_bytes(p) / sizeof(v4u));
      const uint32_t blocks = uint32_t(std::min((words + 255) / 256, int64_t(1024))) + (p.per_sequence ? 0 : 1);
      hipLaunchKernelGGL(gated_clear_kernel, dim3(blocks), dim3(256), 0, stream, *g, p, zeros, words, rows,
                         runs_of(sizeof(T)));
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    choose_streams(*g, KIND, back, sizeof(T), &p);
    const bool ragged = g->channels % (16 / int(sizeof(T))) != 0;
    if (walk) {
      if (ragged) launch_mode<T, KIND, true, kWalk>(*g, p, back, stream);
      else launch_mode<T, KIND, false, kWalk>(*g, p, back, stream);
    } else if (p.sharing) {
      if (ragged) launch_mode<T, KIND, true, kShort>(*g, p, back, stream);
      else launch_mode<T, KIND, false, kShort>(*g, p, back, stream);
    } else {
      if (ragged) launch_mode<T, KIND, true, kTile>(*g, p, back, stream);
      else launch_mode<T, KIND, false, kTile>(*g, p, back, stream);
    }
    return hipGetLastError();
  }
};
template <typename T, int KIND>
struct Step {
  static hipError_t run(float* state, const void* gate, const void* u, void* h, int64_t n, hipStream_t stream) {
    const int64_t blocks = std::min((n + 256 * kStep - 1) / (256 * kStep), int64_t(1) << 20);
    hipLaunchKernelGGL((gated_step_kernel<T, KIND>), dim3(uint32_t(blocks)), dim3(256), 0, stream, state,
                       static_cast<const T*>(gate), static_cast<const T*>(u), static_cast<T*>(h), n);
    return hipGetLastError();
  }
};

}  // namespace

size_t gated_workspace_bytes(int32_t sequences, int64_t tokens, int32_t channels, bool packed) {
  Plan p = {};
  if (!plan_sizes(sequences, tokens, channels, packed, kFewestRows, runs_of(4), &p)) return 0;
  return p.chained ? ticket_bytes(p) + table_bytes(p) + short_bytes(sequences, p) + map_bytes(p) : 256;
}

hipError_t launch_gated_scan(const GatedArgs& a, hipStream_t stream) {
  return dispatch<Scan>(a.dtype, a.gate_kind, &a, false, stream);
}
hipError_t launch_gated_backward(const GatedArgs& a, hipStream_t stream) {
  return dispatch<Scan>(a.dtype, a.gate_kind, &a, true, stream);
}
hipError_t launch_gated_step(int32_t dtype, int32_t gate_kind, float* state, const void* gate, const void* u, void* h,
                             int64_t n, hipStream_t stream) {
  return dispatch<Step>(dtype, gate_kind, state, gate, u, h, n, stream);
}

}  // namespace ssdq
