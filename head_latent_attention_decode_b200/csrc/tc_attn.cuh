// Absorbed split-KV decode attention on tcgen05 for kv_lora_rank 512 and
// qk_rope 64 (the DeepSeek MLA latent), bf16 cache with blocks of a multiple
// of 64 rows.
//
// Persistent and balanced: the batch's 64-row cache tiles, sequence after
// sequence, form one list, and 2-CTA cluster c takes the c-th equal slice of
// it (so every SM pair streams the same number of tiles whatever the context
// lengths). The part of a sequence inside one slice is a segment; each
// segment leaves one split partial (unnormalised O, reference max, sum), and
// attn_combine_kernel merges a sequence's segments.
//
// Per tile: all heads of the token form the MMA's M = 128 rows (fewer heads
// are padded with zeros). CTA r owns latent columns [256 r, 256 r + 256) of
// every tile and the 64 rotary columns of the tiles with odd-even index r:
//   S_r = [q_abs | q_pe]_r . tile_r^T      (tcgen05, M 128 x N 64, K 256 or 320;
//                                          the latent part of Q lives in TMEM,
//                                          q_pe in shared memory; two S buffers)
//   S   = S_r + S_peer                     (the partials swap through DSMEM in
//                                          f16, into two alternating buffers)
//   online softmax, two threads per head (each half of the tile's 64 columns;
//   the halves' maxima meet in shared memory), with a lazily moved reference
//   max: the accumulator is rescaled only when a head's max grows by more than
//   2^8; P (bf16) is written over the peer partial it was computed from, in
//   the MMA's operand layout
//   O_r += P . V_r                         (tcgen05, A = P from shared memory,
//                                          M 128 x N 256, K 64; V = the same
//                                          shared-memory tile read MN-major)
// Every cache byte is read from HBM once and O (128 x 512 fp32) is split over
// the two CTAs' TMEM. A tile's latent stage is held from its load until its
// P.V, its rotary block (every other tile) only until its S, so the latent
// blocks have a 4-deep ring and the rotary blocks 3 slots of their own. S
// alternates between two TMEM buffers, so S(i + 1) runs, and its partial
// crosses to the peer, while the softmax still works on S(i). Warps 0-7 run
// the softmax (warp w: TMEM lane quarter w % 4, column half w / 4), warp 8
// issues TMA, warp 9 the score MMAs and warp 14 the P.V MMAs (one thread each,
// so a P.V never waits behind the issue of a later S), and warps 10-13 send
// each tile's partial scores to the peer as soon as S lands.
//
// FLAT: the schedule begins with n_pre entries that are not sequences but blocks
// of 128 query rows of any sequences, all against one block table (a shared
// prefix); the sequences' own rows follow in the same list, so that one launch
// with one start-up and one tail takes both. The partials are packed.
// C8: the cache is 8-bit (cache8.cuh). TMA brings the CTA's 256 codes of each
// row (16 KB a tile, two raw buffers) and the row scales 2^k_j; four more warps
// widen them to f16, one conversion for two codes, into the latent stage. Codes
// and scales together do not fit f16's exponents, but a tile's rows relative to
// its largest do: with kt the tile's largest k_j less 6 the stage holds
//   V'_j = 2^(k_j - kt) code_j, at most 2^15,
// exact for rows down to 2^-21 of the tile's largest scale (the values of smaller
// ones are off by up to 2^-22 of it), and the rotary rows take 2^-kt as well. Partial scores leave the MMA as S 2^-kt and are brought back to
// real units as they are read; with the reference R of y = score log2(e) + kt the
// weights 2^(y - R) bring V' back to the rows' own size in O, and the row sums take
// them times 2^-kt: one number a tile, so the softmax is the 16-bit cache's. The
// weights are f16 too: kept below 2^15, they hold their 11 bits down to 2^-29 of
// the largest and are off by 2^-40 of it below. So is the query (within +-65504; an
// entry below 2^-14 is off by 2^-25).
// For 64 sequences of 1024 to 16384 rows and 128 heads: 236 us (the 16-bit cache's
// tiles 2400 cycles, these 2650: the three stages, each held from its conversion
// through S, the exchange and the softmax to its P.V, bound it). Widening to bf16,
// scale and all, took three times the instructions and 340 us; scales kept out of V'
// cost the softmax two products a weight and took 424, when this form took 331; smaller
// code then gave 262 (mbar_poll_long), shorter starts, ends and waits the rest.
// Feeding the codes to kind::f8f6f4 MMAs would take as many MMAs, query and weights
// being split in two there, and put their splitting into the softmax.
// The latent ring is three deep, in the same shared memory.
#pragma once

#include "cache8.cuh"
#include "tc_common.cuh"

namespace mla {
namespace tc {

struct TcAttnArgs {
  int n, H, splits, chunk;
  int bs, n_blocks, mbps, max_ctx;
  const int* block_table;
  const int* ctx;
  const bf16* q_abs;   // [n, H, 512]
  int lat_col0, rope_col0;
  float scale_log2;
  float* part_o;   // [n, splits, H, 512]
  float* part_ml;  // [n, splits, H, 2], and the same again at part_ml + ml_r
  int* flag;
  // CTA r of the pair stores its own (m, l) at part_ml + r * ml_r. The two
  // CTAs add the same two partial scores in a different rounding (own fp32 +
  // peer f16), so each half of the latent is normalised with its own statistics.
  long long ml_r;
  // balanced schedule (head-major kernel): `units` clusters, each a slice of at
  // least `min_per` tiles (which keeps every sequence within `splits` segments);
  // nseg[b] receives the number of segments (split partials) of sequence b
  const bf16* q_pe;   // [n, H, 64]
  int units, min_per;
  int* nseg;
  int allow_empty;   // a context length of 0 is valid (the sequence has keys elsewhere)
  // FLAT: n entries, of which entry b < n_pre is the 128 query rows 128 b .. of
  // rows_total against the fixed_len rows of `pre_table`, and entry n_pre + t is
  // sequence t. Cluster c's partial of entry b is unit c + b of [units + n] units of
  // 128 query rows; seg[b] = {first cluster, clusters}
  int n_pre;
  long long rows_total;
  int fixed_len;
  const int* pre_table;
  int2* seg;
  // LSE (the log-sum-exp is wanted): CTA 0 adds the partial scores that CTA 1 rounded to f16, off by d_j;
  // its sum is off by sum_j p_j d_j to first order, which CTA 1 can sum up:
  // corr[unit, row] = sum_j p_j d_j / sum_j p_j. Of the log-sum-exp, 2.9e-5 without it, 1.0e-7 with it
  // (64 sequences of 1024 to 16384 rows, 8-bit, 128 heads), at 339 us instead of 236; the few-head kernel,
  // whose sums are exact, takes 438. An instantiation of its own: in the others its code cost 7 %.
  float* corr;
  // C8: the cache, its blocks' size and where their scales begin
  const uint8_t* c8;
  long long c8_block, c8_scales;
};

constexpr int ATT_NRP = 3;                      // rotary slots (the tiles of this CTA's parity)
constexpr int ATT_THREADS = 480;                // 8 softmax, 1 TMA, 1 S-MMA, 4 sender, 1 P.V-MMA warps
constexpr int ATT_THREADS8 = 608;               // C8: and 4 that widen the codes
constexpr int ATT_MAX_SEQ = 256;                // sequences per call (the prefix table in shared memory)
template <bool C8>
struct AttnSmemT {
  static constexpr int NST = C8 ? 3 : 4;        // latent ring depth
  static constexpr int STAGE = 4 * 8192;        // the 4 latent k-blocks of [64 rows x 64 cols] bf16
  static constexpr int TILE_OFF = 0;
  static constexpr int RAW_OFF = NST * STAGE;   // C8: 2 x 64 rows x 256 codes, [octet][2 k-blocks][8 rows][128 B]
  static constexpr int ROPE_OFF = 4 * STAGE;                // ATT_NRP x [64 x 64] bf16 rotary blocks
  static constexpr int QPE_OFF = ROPE_OFF + ATT_NRP * 8192;   // [128 x 64] bf16 q_pe (MMA operand layout)
  static constexpr int X_OFF = QPE_OFF + 16384;   // 2 x [128 x 64] f16 peer partial S, then P (bf16) over it
  static constexpr int STG_OFF = X_OFF + 32768;   // [128 x 64] f16, our partial on its way out
  static constexpr int RED_OFF = STG_OFF + 16384; // [2 tiles][2 halves][128] fp32 half-row maxima, then [128] l and [128] corr
  static constexpr int PREF_OFF = RED_OFF + 2 * 2 * 128 * 4 + 2 * 128 * 4;   // [ATT_MAX_SEQ + 1] tile prefix sums
  static constexpr int SC_OFF = PREF_OFF + (ATT_MAX_SEQ + 4) * 4;        // C8: row scales [2][64]
  static constexpr int BAR_OFF = SC_OFF + (C8 ? 512 + 16 : 0);
  static constexpr int SIZE = 1024 + BAR_OFF + 512;
  static_assert(SIZE <= 227 * 1024, "shared memory per CTA");
  static_assert(SC_OFF % 16 == 0, "bulk copies");
};
using AttnSmem = AttnSmemT<false>;
// TMEM columns: Q latent [0,128) (bf16 pairs), S buffers [128,192) [192,256), O [256,512)
constexpr uint32_t ATT_TM_Q = 0, ATT_TM_S = 128, ATT_TM_O = 256;

// FLAT: an entry of `rows` query rows counts as this many tiles more than it has when the list is cut,
// about what a segment's start and end cost (query in, O out), or a cluster with many short sequences
// finishes last (32 sequences of up to 1024 rows behind a prefix of 16384, 128 heads: 308 us at 2 for
// every entry, 260 at 4, 217 at 7, 219 at 11; 16 heads, whose own rows start and end sooner, 64 of up to
// 512 behind 8192: 67, 64, 68, 74 us, and 55 with 6 for a prefix block and 3 for them).
__host__ __device__ constexpr int att_pad(int rows) { return 3 + 3 * rows / 128; }

// Walks a cluster's slice of the batch's tile list: sequence b, its tile lt.
template <bool FLAT>
struct TileWalkT {
  const int* pref;   // pref[b] = tiles of entries 0..b-1, each with its padding (shared memory)
  int n, n_pre, pad_own, b, lt;
  __device__ int pad(int e) const { return !FLAT ? 0 : (e < n_pre ? att_pad(128) : pad_own); }
  __device__ int tiles() const { return pref[b + 1] - pref[b] - pad(b); }
  __device__ void enter(int e) {
    b = e;
    lt = 0;
    while (b < n && tiles() == 0) ++b;
  }
  // `k` tiles on (the list is long enough), entry by entry
  __device__ void skip(int k) {
    for (int left = tiles() - lt; k >= left; left = tiles()) {
      k -= left;
      enter(b + 1);
    }
    lt += k;
  }
  __device__ bool seg_last() const { return lt + 1 == tiles(); }
  __device__ void next() {
    if (seg_last()) enter(b + 1);
    else ++lt;
  }
};

// Context length of entry b as the schedule counts it (0 when invalid).
template <bool FLAT = false>
__device__ __forceinline__ int attn_seq_len(const TcAttnArgs& a, int b) {
  if (FLAT) {
    if (b < a.n_pre) return a.fixed_len;
    const int L = a.ctx[b - a.n_pre];
    return (L < 1 || L > a.max_ctx || (long long)L > (long long)a.mbps * a.bs) ? 0 : L;
  }
  const int L = a.ctx[b];
  return (L < 1 || L > a.max_ctx || L > a.mbps * a.bs) ? 0 : L;
}
// Its row of block ids.
template <bool FLAT>
__device__ __forceinline__ const int* attn_table(const TcAttnArgs& a, int b) {
  if (!FLAT) return a.block_table + (long long)b * a.mbps;
  return b < a.n_pre ? a.pre_table : a.block_table + (long long)(b - a.n_pre) * a.mbps;
}
// Its first query row, and how many it has (at most 128).
template <bool FLAT>
__device__ __forceinline__ long long attn_row0(const TcAttnArgs& a, int b) {
  return FLAT && b < a.n_pre ? b * 128LL : (long long)(FLAT ? b - a.n_pre : b) * a.H;
}
template <bool FLAT>
__device__ __forceinline__ int attn_rows(const TcAttnArgs& a, int b) {
  return FLAT && b < a.n_pre ? (int)min(128LL, a.rows_total - b * 128LL) : a.H;
}

// The balanced schedule: the prefix sum of the batch's tiles of 64 rows, in shared
// memory (pref[b] = tiles of entries 0..b-1 with their padding, n + 1 entries, n <=
// 256), and the slice of the flattened tile list that cluster c takes (slices of
// `per`, at least a.min_per): its tiles N, and the first one's entry b0 and place
// lt0 in it, which one warp finds while it has the list in registers. Block 0 of the
// grid writes each entry's segments to a.nseg or a.seg. Every thread of the CTA
// calls it; there is a __syncthreads in it.
struct AttnSlice { int per, N, b0, lt0; };
template <bool FLAT>
__device__ __forceinline__ AttnSlice attn_schedule(const TcAttnArgs& a, int* pref, int c, uint32_t r, int warp, int lane) {
  int* out = pref + ATT_MAX_SEQ + 1;   // N, b0, lt0
  auto pad = [&](int b) { return !FLAT ? 0 : (b < a.n_pre ? att_pad(128) : att_pad(a.H)); };
  if (warp == 0) {
    int cnt[8], sum = 0;   // tiles of entries 8 lane + k
#pragma unroll
    for (int k = 0; k < 8; ++k) cnt[k] = 8 * lane + k < a.n ? attn_seq_len<FLAT>(a, 8 * lane + k) : 0;   // loads in flight
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int b = 8 * lane + k;
      if (b < a.n) {
        if (cnt[k] == 0 && c == 0 && r == 0 && !(a.allow_empty && a.ctx[FLAT ? b - a.n_pre : b] == 0)) set_flag(a.flag, MLA_FLAG_BAD_CONTEXT);
        cnt[k] = (cnt[k] + 63) / 64;
        sum += cnt[k] + pad(b);
      }
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const int total = __shfl_sync(0xffffffffu, incl, 31);   // the batch's tile count
    const int per = max((total + a.units - 1) / a.units, a.min_per), g0 = c * per, g1 = min(total, g0 + per);
    int run = incl - sum, N = 0, b0 = -1, lt0 = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int b = 8 * lane + k;
      if (b < a.n) {
        pref[b] = run;
        const int lo = max(g0, run), n_here = min(g1, run + cnt[k]) - lo;   // its tiles within [g0, g1)
        if (n_here > 0) {
          if (b0 < 0) { b0 = b; lt0 = lo - run; }
          N += n_here;
        }
        run += cnt[k] + pad(b);
      }
    }
    const uint32_t has = __ballot_sync(0xffffffffu, b0 >= 0);
    if (has && lane == __ffs(has) - 1) { out[1] = b0; out[2] = lt0; }
    N = __reduce_add_sync(0xffffffffu, N);
    if (lane == 0) out[0] = N;
    if (lane == 31) pref[a.n] = total;
  }
  __syncthreads();
  const int total = pref[a.n], per = max((total + a.units - 1) / a.units, a.min_per);
  if (blockIdx.x == 0) {   // segments of each entry, for the merge
    for (int b = threadIdx.x; b < a.n; b += blockDim.x) {
      const int T = pref[b + 1] - pref[b] - pad(b);
      const int first = pref[b] / per, last = (pref[b] + T - 1) / per;
      if (FLAT) a.seg[b] = T > 0 ? make_int2(first, last - first + 1) : make_int2(0, 0);
      else a.nseg[b] = T > 0 ? last - first + 1 : 0;
    }
  }
  return {per, out[0], out[1], out[2]};
}

// Two bf16 in f16 (infinite beyond 65504, off by 2^-25 below 2^-14).
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w) {
  const __half2 v = __floats2half2_rn(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return *reinterpret_cast<const uint32_t*>(&v);
}

// The MMA warps' steps, by one lane or (W) by the whole warp with one lane elected (mma_bf16_w). With the
// 15 warps of the 16-bit kernel one lane does better (V3 decode step 0.385 against 0.401 ms: the other
// lanes' polling costs more than the operands' moves), with the 19 of the 8-bit one the whole warp (324
// against 339 us for 128 x 16 query rows over 32767 rows).
template <bool W>
__device__ __forceinline__ bool issue_wait(uint32_t bar, uint32_t parity, volatile int* abort_word, int* flag) {
  return W ? mbar_poll_warp(bar, parity, abort_word, flag) : mbar_wait(bar, parity, abort_word, flag);
}
template <bool W>
__device__ __forceinline__ void issue_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if (W) mma_bf16_ts_w(d, a, b, idesc, acc);
  else mma_bf16_ts(d, a, b, idesc, acc);
}
template <bool W>
__device__ __forceinline__ void issue_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if (W) mma_bf16_w(d, a, b, idesc, acc);
  else mma_bf16(d, a, b, idesc, acc);
}
template <bool W>
__device__ __forceinline__ void issue_commit(uint32_t bar) {
  if (W) mma_commit_w(bar);
  else mma_commit(bar);
}
template <bool W>
__device__ __forceinline__ void issue_commit_mask(uint32_t bar, uint16_t mask) {
  if (W) mma_commit_cta_mask_w(bar, mask);
  else mma_commit_cta_mask(bar, mask);
}

template <bool FLAT, bool C8 = false, bool LSE = false>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(C8 ? ATT_THREADS8 : ATT_THREADS, 1)
    tc_attn_decode_kernel(const __grid_constant__ CUtensorMap tm_cache, const __grid_constant__ CUtensorMap tm_lat,
                          TcAttnArgs a) {
  using SM = AttnSmemT<C8>;
  constexpr int ATT_NST = SM::NST;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t tile_s = sbase + SM::TILE_OFF, x_s = sbase + SM::X_OFF;
  float* red = (float*)(smem + SM::RED_OFF);      // [tile & 1][half][head]
  float* red_l = red + 2 * 2 * 128;                // [head]: the second half's row sum
  int* pref = (int*)(smem + SM::PREF_OFF);
  const uint32_t bar = sbase + SM::BAR_OFF;
  // barriers (8 B each)
  const uint32_t full_b = bar;                        // [ATT_NST] tile landed
  const uint32_t empty_b = bar + 8 * ATT_NST;         // [ATT_NST] tile consumed by P.V
  const uint32_t s_full = bar + 16 * ATT_NST;         // [2] S_r(i) complete, in buffer i & 1
  const uint32_t s_free = s_full + 16;                // [2] S read by the 8 softmax and 4 sender warps
  const uint32_t p_full_b = s_free + 16;              // [2] P(i) in shared memory (8 softmax warps)
  const uint32_t x_full_b = p_full_b + 16;            // [2 buffers][4 lane quarters] peer partial rows landed
  const uint32_t x_free_b = x_full_b + 64;            // [2] the peer's P.V has released its buffer
  const uint32_t q_ready = x_free_b + 16;             // Q of the next segment in TMEM (8 softmax warps)
  const uint32_t o_done = q_ready + 8;                // each P.V
  const uint32_t o_seg = o_done + 8;                  // the last P.V of a segment
  const uint32_t o_free = o_seg + 8;                  // O of a segment read out (8 softmax warps)
  const uint32_t fin = o_free + 8;
  const uint32_t xch_b = fin + 8;                     // [4 quarters][2] the two halves' maxima posted
  const uint32_t l_done = xch_b + 64;                 // [4] the second half's row sums posted
  const uint32_t rope_empty = l_done + 32;            // [ATT_NRP] rotary block consumed by S
  const uint32_t rope_full = rope_empty + 8 * ATT_NRP;   // C8: [ATT_NRP] rotary block landed
  const uint32_t raw_full = rope_full + 8 * ATT_NRP;     // C8: [2] codes and scales landed
  const uint32_t raw_empty = raw_full + 16;              // C8: [2] codes converted
  // of the tile in each stage: rows that count + 128 for a segment's last, its entry; C8: the same of
  // the tile in each raw buffer, and the tiles' kt. The senders read kt too, and no wait of this CTA
  // holds a stage for them: tile t + 8 is converted after this CTA's P.V(t + 5), so after the peer's
  // S(t + 5) and its P.V(t + 2), which took what the senders sent of t.
  int2* tile_of = (int2*)(smem + SM::BAR_OFF + 464);
  int* tile_kt = (int*)(smem + SM::BAR_OFF + 416);   // [8]
  int2* raw_of = (int2*)(smem + SM::SC_OFF + 512);
  uint32_t* tmem_slot = (uint32_t*)(smem + SM::BAR_OFF + 448);
  volatile int* abort_word = (volatile int*)(smem + SM::BAR_OFF + 452);

  const uint32_t r = cluster_ctarank(), peer = r ^ 1u;
  const int c = blockIdx.x >> 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < ATT_NST; ++i) { mbar_init(full_b + 8 * i, C8 ? 4 : 1); mbar_init(empty_b + 8 * i, 1); }
    if (C8) {
      for (int i = 0; i < ATT_NRP; ++i) mbar_init(rope_full + 8 * i, 1);
      for (int i = 0; i < 2; ++i) { mbar_init(raw_full + 8 * i, 1); mbar_init(raw_empty + 8 * i, 4); }
    }
    // S: its MMAs and the issuing thread, which has seen the tile land and with it what the tile is
    for (int i = 0; i < 2; ++i) { mbar_init(s_full + 8 * i, 2); mbar_init(s_free + 8 * i, 12); }
    for (int i = 0; i < ATT_NRP; ++i) mbar_init(rope_empty + 8 * i, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(p_full_b + 8 * i, 8);
      for (int k = 0; k < 4; ++k) mbar_init(x_full_b + 8 * (4 * i + k), 1);
      mbar_init(x_free_b + 8 * i, 1);
    }
    mbar_init(q_ready, 8);
    mbar_init(o_done, 1);
    mbar_init(o_seg, 1);
    mbar_init(o_free, 8);
    mbar_init(fin, 2);   // both issuing threads' last commits
    for (int i = 0; i < 8; ++i) mbar_init(xch_b + 8 * i, 2);
    for (int i = 0; i < 4; ++i) mbar_init(l_done + 8 * i, 1);
    *abort_word = 0;
    fence_mbar_init();
  }
  if (threadIdx.x == 256) {
    prefetch_tmap(&tm_cache);
    prefetch_tmap(&tm_lat);
  }
  __syncthreads();
  cluster_sync_all();   // both CTAs' barriers exist before any remote arrive
  griddep_wait();       // the inputs all come from the stream's earlier kernels, and those may still need their TMEM
  if (warp == 1) { tmem_alloc(smem_u32(tmem_slot), 512); tmem_relinquish(); }
  tc_fence_before();

  // ---- the schedule: tile prefix over the batch, then this cluster's slice ----
  const AttnSlice slice = attn_schedule<FLAT>(a, pref, c, r, warp, lane);
  const int per = slice.per, N = slice.N;
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  using TileWalk = TileWalkT<FLAT>;
  const TileWalk wl{pref, a.n, a.n_pre, att_pad(a.H), slice.b0, slice.lt0};   // at the first tile
  if (N <= 0) {   // both CTAs of the cluster take this branch together
    if (warp == 1) tmem_dealloc(tmem, 512);
    return;
  }
  if (threadIdx.x == 0) griddep_launch_dependents();

  if (warp == 8) {
    // ---------------- TMA producer (lane 0 issues; lane k holds the block id of tile i + k) ----------------
    TileWalk w = wl;
    int i = 0, blkv = 0;
    int2 ofv = make_int2(0, 0);
    for (; i < N; ++i, w.next()) {
      if ((i & 31) == 0) {   // the block ids of the next 32 tiles, loaded in parallel
        TileWalk wk = w;
        if (i + lane < N) {
          wk.skip(lane);
          blkv = attn_table<FLAT>(a, wk.b)[(64 * wk.lt) / a.bs];
          const bool good = blkv >= 0 && blkv < a.n_blocks;
          ofv.x = (good ? min(64, attn_seq_len<FLAT>(a, wk.b) - 64 * wk.lt) : 0) + (i + lane == N - 1 || wk.seg_last() ? 128 : 0);
          ofv.y = wk.b;
        }
      }
      const int blk = __shfl_sync(0xffffffffu, blkv, i & 31);
      const int2 of = make_int2(__shfl_sync(0xffffffffu, ofv.x, i & 31), __shfl_sync(0xffffffffu, ofv.y, i & 31));
      if (FLAT && w.lt == 0 && i > 0) {   // another entry: its query into L2 ahead of the softmax warps
        const long long q0 = attn_row0<FLAT>(a, w.b);
        for (int x = lane; x < attn_rows<FLAT>(a, w.b); x += 32) {
          const char* qa = (const char*)(a.q_abs + (q0 + x) * 512 + 256 * r);
          for (int k = 0; k < 4; ++k) prefetch_l2(qa + 128 * k);
          prefetch_l2(a.q_pe + (q0 + x) * 64);
        }
      }
      const int st = i % ATT_NST;
      const bool rope = (i & 1) == (int)r;
      const int ri = (i >> 1) % ATT_NRP;
      if (C8 ? !mbar_poll_warp(raw_empty + 8 * (i & 1), ((i >> 1) & 1) ^ 1, abort_word, a.flag)
             : !mbar_poll_warp(empty_b + 8 * st, ((i / ATT_NST) & 1) ^ 1, abort_word, a.flag))
        break;
      if (rope && !mbar_poll_warp(rope_empty + 8 * ri, (((i >> 1) / ATT_NRP) & 1) ^ 1, abort_word, a.flag)) break;
      if (C8) {
        if (lane == 0) {
          const int j0 = 64 * w.lt, off = j0 % a.bs, rb = i & 1;
          const bool good = blk >= 0 && blk < a.n_blocks;
          if (!good && r == 0) set_flag(a.flag, MLA_FLAG_BAD_BLOCK);
          const int cur = good ? blk : max(a.n_blocks, 1);   // a block beyond the map: the load fills zeros
          raw_of[rb] = of;
          mbar_arrive_expect_tx(raw_full + 8 * rb, 16384 + (good ? 256 : 0));
          tma_load_5d(sbase + SM::RAW_OFF + rb * 16384, &tm_lat, raw_full + 8 * rb, 0, 0, 2 * (int)r, good ? off / 8 : 0, cur);
          if (good) bulk_load(sbase + SM::SC_OFF + rb * 256, a.c8 + cur * a.c8_block + a.c8_scales + off * 4, 256, raw_full + 8 * rb);
          if (rope) {
            mbar_arrive_expect_tx(rope_full + 8 * ri, 8192);
            tma_load_3d(sbase + SM::ROPE_OFF + ri * 8192, &tm_cache, rope_full + 8 * ri, 0, good ? off : 0, cur);
          }
        }
        continue;
      }
      if (lane == 0) {
        const int j0 = 64 * w.lt;
        long long row = -64;
        if (blk >= 0 && blk < a.n_blocks) row = (long long)blk * a.bs + (j0 % a.bs);
        else if (r == 0) set_flag(a.flag, MLA_FLAG_BAD_BLOCK);
        tile_of[st] = of;
        mbar_arrive_expect_tx(full_b + 8 * st, rope ? 5 * 8192 : 4 * 8192);
        const uint32_t dst = tile_s + st * SM::STAGE;
        // the 4 latent k-blocks of the 64 rows in one box: [8 row octets][4 k-blocks][8 rows][128 B]
        tma_load_4d(dst, &tm_lat, full_b + 8 * st, 0, 0, a.lat_col0 / 64 + 4 * (int)r, (int)(row / 8));
        if (rope) tma_load_3d(sbase + SM::ROPE_OFF + ri * 8192, &tm_cache, full_b + 8 * st, a.rope_col0, (int)row, 0);
      }
    }
    // drain the loads still in flight
    if (C8 && lane == 0) {
      for (int u = (i > 2 ? i - 2 : 0); u < i; ++u) {
        const uint64_t t1 = global_timer_ns();
        while (!mbar_try_wait(raw_full + 8 * (u & 1), (u >> 1) & 1))
          if (global_timer_ns() - t1 > WAIT_LIMIT_NS) { set_flag(a.flag, MLA_FLAG_WAIT_TIMEOUT); break; }
      }
      const int nr = (i + 1 - (int)r) >> 1;   // rotary blocks loaded
      for (int u = (nr > ATT_NRP ? nr - ATT_NRP : 0); u < nr; ++u) {
        const uint64_t t1 = global_timer_ns();
        while (!mbar_try_wait(rope_full + 8 * (u % ATT_NRP), (u / ATT_NRP) & 1))
          if (global_timer_ns() - t1 > WAIT_LIMIT_NS) { set_flag(a.flag, MLA_FLAG_WAIT_TIMEOUT); break; }
      }
    }
    if (!C8 && lane == 0) {
      for (int u = (i > ATT_NST ? i - ATT_NST : 0); u < i; ++u) {
        const uint64_t t1 = global_timer_ns();
        while (!mbar_try_wait(full_b + 8 * (u % ATT_NST), (u / ATT_NST) & 1))
          if (global_timer_ns() - t1 > WAIT_LIMIT_NS) { set_flag(a.flag, MLA_FLAG_WAIT_TIMEOUT); break; }
      }
    }
  } else if (warp == 9) {
    // ---------------- S issuer: S(t) into buffer t & 1 once its tile has landed ----------------
    if (C8 || lane == 0) {   // C8: the whole warp runs the loop
      constexpr uint32_t idesc_s = C8 ? idesc_f16(128, 64) : idesc_bf16(128, 64), idesc_pe = idesc_bf16(128, 64);
      // descriptors built once; stages and k-steps add their byte offset >> 4
      const uint64_t d_t = sdesc_sw128_sbo(tile_s, 4096), d_rope = sdesc_sw128(sbase + SM::ROPE_OFF);
      const uint64_t d_qpe = sdesc_sw128(sbase + SM::QPE_OFF);
      TileWalk ws = wl;
      int ks = 0;
      for (int t = 0; t < N; ++t, ws.next()) {
        const int st = t % ATT_NST;
        const bool first = (t == 0 || ws.lt == 0), last = (t == N - 1 || ws.seg_last());
        if (!issue_wait<C8>(full_b + 8 * st, (t / ATT_NST) & 1, abort_word, a.flag) ||
            !issue_wait<C8>(s_free + 8 * (t & 1), ((t >> 1) & 1) ^ 1, abort_word, a.flag) ||
            (first && !issue_wait<C8>(q_ready, ks & 1, abort_word, a.flag)))
          break;
        tc_fence_after();
        const uint64_t dt = d_t + (uint64_t)(st * (SM::STAGE / 16));
        const uint32_t d = tmem + ATT_TM_S + 64 * (t & 1);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            issue_ts<C8>(d, tmem + ATT_TM_Q + 32 * j + 8 * k, dt + (j * 1024 + 32 * k) / 16, idesc_s,
                        (j > 0 || k > 0) ? 1u : 0u);
        if ((t & 1) == (int)r) {
          const int ri = (t >> 1) % ATT_NRP;
          const uint64_t dr = d_rope + (uint64_t)(ri * (8192 / 16));
#pragma unroll
          for (int k = 0; k < 4; ++k) issue_ss<C8>(d, d_qpe + 2 * k, dr + 2 * k, idesc_pe, 1u);
          issue_commit<C8>(rope_empty + 8 * ri);
        }
        issue_commit<C8>(s_full + 8 * (t & 1));
        if (lane == 0) mbar_arrive(s_full + 8 * (t & 1));
        if (last) ++ks;
      }
      issue_commit<C8>(fin);
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(fin, 0))
        if (global_timer_ns() - t0 > WAIT_LIMIT_NS) { set_flag(a.flag, MLA_FLAG_WAIT_TIMEOUT); break; }
    }
  } else if (warp == 14) {
    // ---------------- P.V issuer: O += P(u) . V(u) as soon as P(u) is written ----------------
    if (C8 || lane == 0) {
      constexpr uint32_t idesc_o = C8 ? idesc_f16(128, 256, 1) : idesc_bf16(128, 256, 1);
      const uint64_t d_v = sdesc_sw128_mn_sbo(tile_s, 1024, 4096), d_p = sdesc_sw128(x_s);
      TileWalk wo = wl;
      int ko = 0;
      for (int u = 0; u < N; ++u, wo.next()) {
        const int st = u % ATT_NST, xb = u & 1;
        const bool first = (u == 0 || wo.lt == 0), last = (u == N - 1 || wo.seg_last());
        if (!issue_wait<C8>(p_full_b + 8 * xb, (u >> 1) & 1, abort_word, a.flag) ||
            (first && ko > 0 && !issue_wait<C8>(o_free, (ko - 1) & 1, abort_word, a.flag)))
          break;
        tc_fence_after();
        const uint64_t dv = d_v + (uint64_t)(st * (SM::STAGE / 16));
        const uint64_t dp = d_p + (uint64_t)(xb * (16384 / 16));
#pragma unroll
        for (int k = 0; k < 4; ++k)
          issue_ss<C8>(tmem + ATT_TM_O, dp + 2 * k, dv + 8192 * k / 16, idesc_o, (!first || k > 0) ? 1u : 0u);
        issue_commit<C8>(o_done);
        issue_commit<C8>(empty_b + 8 * st);
        issue_commit_mask<C8>(x_free_b + 8 * xb, (uint16_t)(1u << peer));   // our buffer xb is the peer's to fill
        if (last) { issue_commit<C8>(o_seg); ++ko; }
      }
      issue_commit<C8>(fin);
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(fin, 0))
        if (global_timer_ns() - t0 > WAIT_LIMIT_NS) { set_flag(a.flag, MLA_FLAG_WAIT_TIMEOUT); break; }
    }
  } else if (C8 && warp > 14) {   // warps 15-18
    // ---------------- C8: tile t's codes -> its f16 stage. This warp takes chunks [4 (cw & 1), +4) of
    // 16 codes of k-block cw >> 1 of every row: lane = row of an octet + 8 x chunk, so that the 128-byte
    // swizzle spreads loads and stores over all banks. Rows that do not count become zeros.
    const int cw = warp - 15, ro = lane & 7, cc = 4 * (cw & 1) + (lane >> 3);
    const int o0 = ((2 * (cc & 3)) ^ ro) << 4, o1 = ((2 * (cc & 3) + 1) ^ ro) << 4;
    for (int t = 0; t < N; ++t) {
      const int rb = t & 1, st = t % ATT_NST;
      if (!mbar_poll_warp(raw_full + 8 * rb, (t >> 1) & 1, abort_word, a.flag)) break;
      const int2 of = raw_of[rb];
      const int rows = of.x & 127;
      const float* sc = reinterpret_cast<const float*>(smem + SM::SC_OFF + rb * 256);
      // the exponents of rows lane and lane + 32 (none: far below every scale), kt, the rows' factors 2^(k - kt)
      auto exponent = [&](int row) {
        const float v = row < rows ? sc[row] : 0.f;
        return v > 0.f ? (int)(__float_as_uint(v) >> 23) - 127 : -1000;
      };
      const int k0 = exponent(lane), k1 = exponent(lane + 32);
      const int km = __reduce_max_sync(0xffffffffu, max(k0, k1)), kt = km > -1000 ? km - 6 : 0;
      auto factor = [&](int k) -> uint32_t {
        const int d = k - kt;
        return d >= -14 ? (uint32_t)(d + 15) << 10 : (d >= -24 ? 1u << (d + 24) : 0u);
      };
      const uint32_t f01 = factor(k0) | factor(k1) << 16;
      if (!mbar_poll_warp(empty_b + 8 * st, ((t / ATT_NST) & 1) ^ 1, abort_word, a.flag)) break;
      if (cw == 0 && lane == 0) { tile_of[st] = of; tile_kt[t & 7] = kt; }
      const uint8_t* src = smem + SM::RAW_OFF + rb * 16384 + (cw >> 1) * 1024 + ro * 128 + ((cc ^ ro) << 4);
      uint8_t* dst = smem + SM::TILE_OFF + st * SM::STAGE + (2 * (cw >> 1) + (cc >> 2)) * 1024 + ro * 128;
#pragma unroll
      for (int oct = 0; oct < 8; ++oct) {
        uint4 cv = *reinterpret_cast<const uint4*>(src + oct * 2048);
        if (8 * oct + ro >= rows) cv = make_uint4(0, 0, 0, 0);
        const uint32_t fb = __byte_perm(__shfl_sync(0xffffffffu, f01, (8 * oct + ro) & 31), 0, oct < 4 ? 0x1010 : 0x3232);
        const __half2 f = *reinterpret_cast<const __half2*>(&fb);
        const uint32_t w[4] = {cv.x, cv.y, cv.z, cv.w};
        uint32_t o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          uint32_t c2;
          asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(c2) : "h"((uint16_t)(w[k >> 1] >> (16 * (k & 1)))));
          const __half2 p = __hmul2(*reinterpret_cast<const __half2*>(&c2), f);
          o[k] = *reinterpret_cast<const uint32_t*>(&p);
        }
        *reinterpret_cast<uint4*>(dst + oct * 4096 + o0) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(dst + oct * 4096 + o1) = make_uint4(o[4], o[5], o[6], o[7]);
      }
      if ((t & 1) == (int)r) {   // the rotary block times 2^-kt, in place
        const int ri = (t >> 1) % ATT_NRP;
        if (!mbar_poll_warp(rope_full + 8 * ri, ((t >> 1) / ATT_NRP) & 1, abort_word, a.flag)) break;
        const __nv_bfloat162 f = __float2bfloat162_rn(exp2_int(-kt));
        uint4* pe = reinterpret_cast<uint4*>(smem + SM::ROPE_OFF + ri * 8192) + 128 * cw + lane;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint4 v = pe[32 * k];
          uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 p = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w[j]), f);
            w[j] = *reinterpret_cast<const uint32_t*>(&p);
          }
          pe[32 * k] = v;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) { mbar_arrive(full_b + 8 * st); mbar_arrive(raw_empty + 8 * rb); }
    }
  } else if (warp >= 10) {   // warps 10-13
    // ---------------- senders: S_r(i) -> staging -> per warp, one bulk copy of its 32 rows into the
    // peer's X, landing on that quarter's barrier (the peer's softmax warps of the quarter wait for it alone)
    const int qs = warp & 3;                              // TMEM lane quarter of this warp
    const int h = 32 * qs + lane;
    const uint32_t lane_base = (uint32_t)(qs * 32) << 16;
    const uint32_t peer_x = mapa_shared(x_s, peer), peer_x_full = mapa_shared(x_full_b, peer);
    const uint32_t stg_s = sbase + SM::STG_OFF + 4096 * qs;   // this warp's rows, 4 KB
    uint4* stg_row = (uint4*)(smem + SM::STG_OFF + h * 128);
    for (int i = 0; i < N; ++i) {
      if (!mbar_poll_warp(s_full + 8 * (i & 1), (i >> 1) & 1, abort_word, a.flag)) break;
      tc_fence_after();
      const float un = C8 ? exp2_int(tile_kt[i & 7]) : 1.f;
      const uint32_t sa = tmem + ATT_TM_S + 64 * (i & 1) + lane_base;
      if (lane == 0) bulk_wait_read_all();               // this warp's previous copy has left its rows
      __syncwarp();
      // the partial goes out in f16 (half the distributed-shared-memory bytes of fp32; the
      // partial scores stay far inside f16's range and its 11-bit significand costs the
      // scores ~1e-3 relative, well inside the output tolerance)
#pragma unroll 1
      for (int k0 = 0; k0 < 8; k0 += 2) {
        float v[16];
        tmem_ld16(sa + 8 * k0, (uint32_t*)v);
        tmem_ld_wait<16>((uint32_t*)v);
#pragma unroll
        for (int k = 0; k < 2; ++k) {  // chunk k0 + k (8 values) of row h at slot (k0 + k) ^ (h & 7): no bank conflicts
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            __half2 hv = C8 ? __floats2half2_rn(v[8 * k + 2 * j] * un, v[8 * k + 2 * j + 1] * un)
                            : __floats2half2_rn(v[8 * k + 2 * j], v[8 * k + 2 * j + 1]);
            w[j] = *reinterpret_cast<uint32_t*>(&hv);
          }
          stg_row[(k0 + k) ^ (h & 7)] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(s_free + 8 * (i & 1));
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        // the peer's P.V(i - 2) has released the buffer we send into
        const int xb = i & 1;
        if (mbar_wait_cluster(x_free_b + 8 * xb, ((i >> 1) & 1) ^ 1, abort_word, a.flag)) {
          bulk_copy_to_peer(peer_x + xb * 16384 + 4096 * qs, stg_s, 4096, peer_x_full + 8 * (4 * xb + qs));
          bulk_commit_group();
        }
      }
    }
    if (lane == 0) bulk_wait_read_all();
  } else {
    // ---------------- softmax: head h <-> TMEM lane h, columns [32 g, 32 g + 32) of each tile ----------------
    const int q = warp & 3, g = warp >> 2;
    const int h = 32 * q + lane;
    const uint32_t lane_base = (uint32_t)(q * 32) << 16;
    // this half's share of sequence b's query: 128 latent values of CTA r's half
    // -> TMEM columns [64 g, 64 g + 64), 32 rotary values -> [128 + 16 g, 128 + 16 g + 16)
    auto load_q = [&](int b) {
      const bool live = h < attn_rows<FLAT>(a, b);
      const long long qh = attn_row0<FLAT>(a, b) + (live ? h : 0);
      const uint4* src = (const uint4*)(a.q_abs + qh * 512 + r * 256 + 128 * g);
      const uint4* pe = (const uint4*)(a.q_pe + qh * 64 + 32 * g);
      const uint4 zero = make_uint4(0, 0, 0, 0);
      uint4 pv[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) pv[k] = live ? pe[k] : zero;
      constexpr int NL = 8;   // loads in flight: their latency is what this costs (all 16: 2 us slower at 16 heads)
#pragma unroll 1
      for (int k0 = 0; k0 < 16; k0 += NL) {
        uint4 v[NL];
#pragma unroll
        for (int k = 0; k < NL; ++k) v[k] = live ? src[k0 + k] : zero;
#pragma unroll
        for (int k = 0; k < NL; k += 4) {
          uint32_t qv[16];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint4 x = v[k + j];
            if (C8) x = make_uint4(bf16x2_to_f16x2(x.x), bf16x2_to_f16x2(x.y), bf16x2_to_f16x2(x.z), bf16x2_to_f16x2(x.w));
            qv[4 * j] = x.x; qv[4 * j + 1] = x.y; qv[4 * j + 2] = x.z; qv[4 * j + 3] = x.w;
          }
          tmem_st16(tmem + ATT_TM_Q + lane_base + 64 * g + 4 * (k0 + k), qv);
        }
      }
      // q_pe row h, chunks 4 g .. 4 g + 3, in the 128-byte-swizzled K-major operand layout
      uint4* qrow = (uint4*)(smem + SM::QPE_OFF + h * 128);
#pragma unroll
      for (int k = 0; k < 4; ++k) qrow[(4 * g + k) ^ (h & 7)] = pv[k];
      fence_proxy_async_smem();
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_ready);
    };
    load_q(wl.b);
    constexpr float above = C8 ? 15.f : 8.f, below = C8 ? 7.f : 0.f;
    float m_ref = -INFINITY, l = 0.f, dl = 0.f;
    int tseg = 0, kseg = 0;   // tile within the segment, segments done
    bool ok = true;
    for (int i = 0; i < N && ok; ++i) {
      const int st = i % ATT_NST, xb = i & 1;
      if (g == 0 && lane == 0) mbar_arrive_expect_tx(x_full_b + 8 * (4 * xb + q), 4096);   // this quarter's rows
      if (!mbar_poll_warp(s_full + 8 * xb, (i >> 1) & 1, abort_word, a.flag)) { ok = false; break; }
      tc_fence_after();
      float v[32];
      const uint32_t sp_addr = tmem + ATT_TM_S + 64 * xb + 32 * g + lane_base;
      tmem_ld16(sp_addr, (uint32_t*)&v[0]);
      tmem_ld16(sp_addr + 16, (uint32_t*)&v[16]);
      const int2 of = tile_of[st];
      const int valid = of.x & 127, b = of.y;
      const bool last = of.x & 128;
      const int kt = C8 ? tile_kt[i & 7] : 0;
      const float un = C8 ? exp2_int(kt) : 1.f;
      tmem_ld_wait<32>((uint32_t*)v);
      tc_fence_before();
      __syncwarp();
      const bool corr = LSE && r == 1;
      if (lane == 0 && !corr) mbar_arrive(s_free + 8 * xb);   // S(i + 2) may overwrite the buffer
      if (!mbar_poll_warp(x_full_b + 8 * (4 * xb + q), (i >> 1) & 1, abort_word, a.flag)) { ok = false; break; }
      // row h, chunks 4 g .. 4 g + 3 of the peer's partial; P(i) later goes to exactly these bytes
      uint4* xrow = (uint4*)(smem + SM::X_OFF + xb * 16384 + h * 128);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint4 x = xrow[(4 * g + k) ^ (h & 7)];
        const uint32_t wx[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&wx[j]));
          const float2 s = make_float2(v[8 * k + 2 * j], v[8 * k + 2 * j + 1]);
          const float2 s2 = C8 ? fma2(s, make_float2(un, un), f) : add2(s, f);
          v[8 * k + 2 * j] = s2.x;
          v[8 * k + 2 * j + 1] = s2.y;
        }
      }
      if (valid < 64) {
        const int vc = valid - 32 * g;   // valid columns of this half
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = (j < vc) ? v[j] : -INFINITY;   // also drops NaN past the context
      }
      float m4[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
      for (int j = 4; j < 28; j += 8)
#pragma unroll
        for (int k = 0; k < 4; ++k) m4[k] = max3(m4[k], v[j + k], v[j + 4 + k]);
#pragma unroll
      for (int k = 0; k < 4; ++k) m4[k] = fmaxf(m4[k], v[28 + k]);
      const float mloc = fmaxf(max3(m4[0], m4[1], m4[2]), m4[3]);
      // the two halves of head h meet: both then take the same decisions
      red[(xb * 2 + g) * 128 + h] = mloc;
      __syncwarp();
      if (lane == 0) mbar_arrive(xch_b + 8 * (2 * q + xb));
      if (!mbar_poll_warp(xch_b + 8 * (2 * q + xb), (i >> 1) & 1, abort_word, a.flag)) { ok = false; break; }
      float mt = fmaxf(mloc, red[(xb * 2 + (g ^ 1)) * 128 + h]) * a.scale_log2;
      if (C8) mt += (float)kt;
      // online softmax in log2 units with a lazily moved reference max
      float alpha = 1.f;
      bool rescale = false;
      if (mt > m_ref + above) {
        if (m_ref != -INFINITY) { alpha = ex2_approx(m_ref + below - mt); rescale = true; }
        m_ref = mt - below;
      }
      float nm = (m_ref == -INFINITY) ? 0.f : -m_ref;
      if (C8) nm += (float)kt;
      const float2 sl2 = make_float2(a.scale_log2, a.scale_log2), nm2 = make_float2(nm, nm);
      float2 ps[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      uint32_t pk[16];
#pragma unroll
      for (int j = 0; j < 32; j += 2) {
        float2 e = fma2(make_float2(v[j], v[j + 1]), sl2, nm2);
        e = make_float2(ex2_approx(e.x), ex2_approx(e.y));
        ps[(j >> 1) & 1] = add2(ps[(j >> 1) & 1], e);
        if (C8) {
          const __half2 pb = __floats2half2_rn(e.x, e.y);
          pk[j >> 1] = *reinterpret_cast<const uint32_t*>(&pb);
        } else {
          const __nv_bfloat162 pb = __floats2bfloat162_rn(e.x, e.y);
          pk[j >> 1] = *reinterpret_cast<const uint32_t*>(&pb);
        }
      }
      const float2 pt = add2(ps[0], ps[1]);
      float psum = pt.x + pt.y;
      if (C8) psum *= exp2_int(-kt);
      if (__any_sync(0xffffffffu, rescale) && tseg >= 1) {
        // P.V(i - 2) is complete (its release let the peer fill this X buffer), so
        // waiting for the phase of P.V(i - 1) cannot pass early; O must not be
        // touched before it completes
        if (!mbar_poll_warp(o_done, (i - 1) & 1, abort_word, a.flag)) { ok = false; break; }
        tc_fence_after();
        for (int k = 0; k < 8; ++k) {
          uint32_t o[16];
          const uint32_t oa = tmem + ATT_TM_O + lane_base + 128 * g + 16 * k;
          tmem_ld16(oa, o);
          tmem_ld_wait<16>(o);
#pragma unroll
          for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
          tmem_st16(oa, o);
        }
        tmem_st_wait();
        tc_fence_before();
      }
      l = l * alpha + psum;
      if (!C8 && valid < 64) {
        // rows past the context may hold anything (even NaN); P is 0 there, but
        // 0 * NaN is not, so clear them in the four latent slots before P.V
        // (latent rows are laid out [8 row octets][4 k-blocks][8 rows][128 B])
        const int ti = g * 128 + h, row = valid + (ti >> 2);
        if (row < 64) {
          uint8_t* rp = smem + SM::TILE_OFF + st * SM::STAGE + (row >> 3) * 4096 + (ti & 3) * 1024 + (row & 7) * 128;
#pragma unroll
          for (int k = 0; k < 8; ++k) *reinterpret_cast<uint4*>(rp + 16 * k) = make_uint4(0, 0, 0, 0);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        xrow[(4 * g + k) ^ (h & 7)] = make_uint4(pk[4 * k], pk[4 * k + 1], pk[4 * k + 2], pk[4 * k + 3]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full_b + 8 * xb);
      if (corr) {   // this CTA's own partial once more: what the peer got of it less what it is, times the weights
        float u[32];
        tmem_ld16(sp_addr, (uint32_t*)&u[0]);
        tmem_ld16(sp_addr + 16, (uint32_t*)&u[16]);
        tmem_ld_wait<32>((uint32_t*)u);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_free + 8 * xb);
        if (valid < 64) {
          const int vc = valid - 32 * g;
#pragma unroll
          for (int j = 0; j < 32; ++j) u[j] = (j < vc) ? u[j] : 0.f;
        }
        float2 ds = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
          const float2 own = make_float2(u[j] * un, u[j + 1] * un);
          const float2 sent = __half22float2(__floats2half2_rn(own.x, own.y));
          const float2 w = C8 ? __half22float2(*reinterpret_cast<const __half2*>(&pk[j >> 1]))
                              : make_float2(__uint_as_float(pk[j >> 1] << 16), __uint_as_float(pk[j >> 1] & 0xFFFF0000u));
          ds = fma2(w, make_float2(sent.x - own.x, sent.y - own.y), ds);
        }
        float d = ds.x + ds.y;
        if (C8) d *= exp2_int(-kt);
        dl = dl * alpha + d;
      }
      ++tseg;
      if (last) {
        // the segment's S MMAs are all complete (the softmax read each S): the next
        // segment's query may replace this one while the last P.V runs
        if (i + 1 < N) {
          TileWalk wn = wl;
          wn.enter(b + 1);
          load_q(wn.b);
        }
        const int j = c - pref[b] / per;               // this segment's split slot in sequence b
        const long long unit = FLAT ? (long long)c + b : (long long)b * a.splits + j;
        const int rows_u = FLAT ? 128 : a.H;
        const bool store = h < attn_rows<FLAT>(a, b);
        float* const ml = a.part_ml + r * a.ml_r;      // this CTA's (m, l) copy
        if (!mbar_poll_warp(o_seg, kseg & 1, abort_word, a.flag)) { ok = false; break; }
        tc_fence_after();
        float* po = a.part_o + (unit * rows_u + h) * 512 + r * 256 + 128 * g;
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {   // whole sectors: 32 bytes of a row per store
          uint32_t o[32];
          tmem_ld16(tmem + ATT_TM_O + lane_base + 128 * g + 32 * k, o);
          tmem_ld16(tmem + ATT_TM_O + lane_base + 128 * g + 32 * k + 16, o + 16);
          tmem_ld_wait<32>(o);
          if (store) {
#pragma unroll
            for (int jj = 0; jj < 32; jj += 8) st_global_8(po + 32 * k + jj, o + jj);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(o_free);   // the next segment's first P.V may overwrite O
        // the row sum is the two halves' sums
        if (g == 1) {
          red_l[h] = l;
          if (LSE) red_l[128 + h] = dl;
          __syncwarp();
          if (lane == 0) mbar_arrive(l_done + 8 * q);
        } else if (mbar_poll_warp(l_done + 8 * q, kseg & 1, abort_word, a.flag)) {
          if (store) {
            ml[(unit * rows_u + h) * 2] = m_ref * 0.69314718055994531f;   // natural-log units
            const float sum = l + red_l[h];
            ml[(unit * rows_u + h) * 2 + 1] = sum;
            if (LSE && r == 1)
              a.corr[unit * 128 + h] = sum > 0.f ? (dl + red_l[128 + h]) * (a.scale_log2 * 0.69314718055994531f) / sum : 0.f;
          }
        } else {
          ok = false;
          break;
        }
        m_ref = -INFINITY;
        l = dl = 0.f;
        tseg = 0;
        ++kseg;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  cluster_sync_all();   // no CTA leaves while its peer may still touch its shared memory
}

}  // namespace tc
}  // namespace mla
