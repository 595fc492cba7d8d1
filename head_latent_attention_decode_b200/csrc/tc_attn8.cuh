// Latent attention over the 8-bit cache on tcgen05 with the DeepSeek latent
// (kv_lora_rank 512, qk_rope 64) and blocks of a multiple of 16 rows: up to 64
// heads, beyond 128, and any number where the blocks are no multiple of 64 rows
// (latent_plan has the rules). The E4M3 codes go to the tensor cores as they are (kind::f8f6f4); no
// value is ever widened in shared memory.
//
// The other operand of each product would lose accuracy in E4M3, so it is split
// in two E4M3 parts, x = hi + lo / m with hi = e4m3(x) and lo = e4m3(m (x - hi)): two
// 4-bit significands carry the 8 bits of a bf16 value, and both parts ride in one MMA
// as extra columns (N = 32 for 16 heads), whose sums only meet in registers. So lo has
// a scale m of its own, the largest power of two that keeps it within E4M3, and with it
// hi's smallest steps divided by m. An MMA of M 128 takes as long as its
// operands' way out of shared memory, 40 cycles for N 32 and 39 for N 16 (48 for
// 64, 63 for 128; K- or MN-major and 8- or 16-bit alike), so the second part is
// nearly free.
//   q_abs_h = 2^k_h (hi + lo / 16): k_h brings the row's largest to at most 448; columns
//     within 2^-14 of it are exact, smaller ones off by at most 2^-22 of it
//   p: relative to a per-head reference R that follows the tiles' maxima both up
//     and down, so that thousands of light keys behind a heavy one keep their
//     weight: a weight hi + lo / 32 is off by 2^-8 of itself or 2^-17 of the largest
//     of the last few tiles (with m = 1 it was 2^-12, and hundreds of keys that light
//     went missing from o while l counted them: 1.5 % of o where the values share a mean)
//
// The row scale s_j = 2^k_j folds into both products: with u_hj = q_h . code_j,
//   y_hj = scale log2(e) (s_j u_hj + q_pe_h . k_pe_j) + k_j
//   w_hj = 2^(y_hj - R_h + 8) in [0, 256],  R_h >= max over the tile's keys of y_hj
//   O_h  = sum_j w_hj code_j  (= 2^(8 - R_h) sum_j p_hj s_j code_j)
//   l_h  = sum_j w_hj 2^-k_j
//
// Transposed tiles as in the 16-bit few-head kernel: 128 cache rows fill the
// MMA's M. One CTA takes whole rows (an 8-bit tile is 64 KB of codes and 16 KB
// of rotary keys, so nothing has to be exchanged between CTAs):
//   U^T [128 keys x (hi | lo)] = codes . Q^T          16 MMAs, M 128 x N 32 x K 32
//   R^T [128 keys x 16]        = k_pe . q_pe^T (bf16)  4 MMAs, M 128 x N 16 x K 16
//   O^T [128 latent x (hi | lo)] x 4 = codes^T . W^T  16 MMAs; codes^T is the same
//                                                     shared-memory tile read MN-major
//
// Two sets of four softmax warps (thread <-> key; for a rescale and at the end
// thread <-> latent column) take the tiles of either parity, each with S, W and
// rotary buffers, an O^T in TMEM, references and row sums of its own. A tile's
// softmax is a chain of short dependent steps, about as long as HBM takes for
// the tile, so two chains run at a time; and as the sets share nothing until an
// entry ends, a set's O^T is at rest when its next tile moves a reference. One
// warp each issues TMA, the score MMAs and the value MMAs. The TMA warp also
// brings the tile's row scales (a bulk copy per box) and writes what the softmax
// has to know of the tile, so that the softmax warps touch no table.
//
// Schedule: the tiles of all entries (sequences; or blocks of 16 query rows
// against one shared prefix) form one list, and each CTA takes an equal slice.
// More than 16 heads: `groups` CTAs, each with 16 heads, walk the same slice at
// the same time, so the rows come from HBM once and from L2 after.
//
// 16 heads, caches cold, by the kernel timer over 1 to 28 tiles an SM: 15 us to
// start and end (lengths, block table, first tile and query each a trip to memory,
// first fetches of code; O out), and 2.3 us a tile (5.3 TB/s of codes, rotary keys
// and scales). 32 sequences of 4096 rows are 7 tiles an SM: 31 us, and 32 a call with
// the merge. 64 sequences of 1024 to 16384 rows, 128 heads in 8 groups: 438 us.
#pragma once

#include "cache8.cuh"
#include "tc_common.cuh"

namespace mla {
namespace tc {

// kind::f8f6f4: fp32 accumulator, A and B E4M3 (format 0).
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, int a_mn_major = 0) {
  return (1u << 4) | ((uint32_t)a_mn_major << 15) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

struct TcAttn8Args {
  int n_ent, groups, units;   // entries; head groups; slices (grid = units x groups)
  int flat;                   // 0: entry e is sequence e, its rows e H + 16 group ..; 1: query rows 16 e .. against one table
  int H;                      // query rows per sequence (flat = 0)
  long long rows_total;       // query rows in all
  const int* ctx;             // lengths (flat = 0)
  int len, min_ctx, max_ctx;  // length (flat = 1); the valid lengths
  const int* table;           // block ids; row e at table + e * table_stride
  long long table_stride;
  int mbps, bs, box, n_blocks;
  const uint8_t* cache;
  long long block_bytes, sc_off;
  const bf16* q_abs;          // [rows_total, 512]
  const bf16* q_pe;           // [rows_total, 64]
  float scale_log2;
  float* part_o;              // [groups][units + n_ent][16][512]: unit c + e of group g
  float* part_ml;             // the same [..][16][2]
  int2* seg;                  // [n_ent]: {first slice, slices} of each entry
  int* flag;
};

constexpr float A8_QLO = 16.f, A8_WLO = 32.f;   // the scales m: |x - hi| <= 16 for |x| <= 448, <= 8 for x <= 256

// Two E4M3 values times m, exact in f16 for a power of two of up to 2^7.
__device__ __forceinline__ float2 e4m3x2_times(uint16_t c, float m) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  return __half22float2(__hmul2(*reinterpret_cast<const __half2*>(&h), __float2half2_rn(m)));
}

constexpr int A8_MAX_ENT = 768;   // sequences per launch (their tile prefix in shared memory)

constexpr int A8_THREADS = 8 * 32 + 96;   // two sets of four softmax warps; TMA, score and value MMA warps
struct Attn8Smem {
  static constexpr int NPR = 5;                   // ring entries of 32 KB: two per tile
  static constexpr int QB = 32 * 128;             // one k-block [32 x 128 B] of Q
  static constexpr int PB = 32 * 128;             // one buffer of W^T [32 x 128 keys]
  static constexpr int RING_OFF = 0;              // entry: [16 row octets][2 k-blocks][8 rows][128 B]
  static constexpr int ROPE_OFF = NPR * 32768;    // 2 x [128 x 64] bf16
  static constexpr int Q_OFF = ROPE_OFF + 2 * 16384;
  static constexpr int QPE_OFF = Q_OFF + 4 * QB;
  static constexpr int P_OFF = QPE_OFF + 16 * 128;
  static constexpr int SC_OFF = P_OFF + 2 * PB;   // row scales [2][128]
  static constexpr int RED_OFF = SC_OFF + 2 * 128 * 4;
  // floats: maxima [2 sets][2][4 warps][16]; query scales [2 entries][16]; posted row sums [4 tiles][4 warps][16]
  // and references [4][16]; per warp 8 - R and the factors of a rescale [2][16]
  static constexpr int RED_SLQ = 256, RED_RL = RED_SLQ + 32, RED_RP = RED_RL + 256, RED_WARP = RED_RP + 64;
  static constexpr int RED_FLOATS = RED_WARP + 8 * 32;
  static constexpr int PREF_OFF = RED_OFF + RED_FLOATS * 4;
  static constexpr int BAR_OFF = PREF_OFF + (A8_MAX_ENT + 4) * 4;
  static constexpr int SIZE = 1024 + BAR_OFF + 512;
  // TMEM: per set S [(hi 8 | lo 8) x 2 | rotary 16], then per set O^T of the four latent groups [(hi 8 | lo 8) x 2]
  static constexpr int TM_S = 0, TM_O = 128;
  static_assert(SIZE <= 227 * 1024, "shared memory per CTA");
  static_assert(BAR_OFF % 16 == 0 && P_OFF % 1024 == 0, "alignment");
};

__device__ __forceinline__ int a8_len(const TcAttn8Args& a, int e) {
  if (a.flat) return a.len;
  const int L = a.ctx[e];
  return (L < a.min_ctx || L > a.max_ctx || (long long)L > (long long)a.mbps * a.bs) ? 0 : L;
}

// Walks a slice of the tile list: entry e, its tile lt, its length and tiles.
struct Walk8 {
  const int* pref;   // tiles before entry e (shared memory), or NULL: e * T
  int T, n, e, lt, len, tiles;
  __device__ __forceinline__ int at(int i) const { return pref ? pref[i] : i * T; }
  __device__ __forceinline__ void enter(const TcAttn8Args& a) {
    len = a8_len(a, e);
    tiles = (len + 127) / 128;
  }
  __device__ __forceinline__ bool seg_last() const { return lt + 1 == tiles; }
  __device__ __forceinline__ void next(const TcAttn8Args& a) {
    if (!seg_last()) { ++lt; return; }
    lt = 0;
    do {
      if (++e == n) { len = tiles = 0; return; }
      enter(a);
    } while (tiles == 0);
  }
};

// What the TMA warp says of a tile: how many tiles of its entry follow in this slice (2: two or
// more), whether it or the tile before it is its entry's first here, and the parity of the entry.
constexpr int TILE_LEFT = 3, TILE_FIRST = 4, TILE_PREV_FIRST = 8, TILE_ODD = 16;

__global__ void __launch_bounds__(A8_THREADS, 1)
    tc_attn8_kernel(const __grid_constant__ CUtensorMap tm_codes, const __grid_constant__ CUtensorMap tm_rope,
                    TcAttn8Args a) {
  using SM = Attn8Smem;
  constexpr int NPR = SM::NPR;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t ring_s = sbase + SM::RING_OFF, rope_s = sbase + SM::ROPE_OFF, q_s = sbase + SM::Q_OFF,
                 qpe_s = sbase + SM::QPE_OFF, p_s = sbase + SM::P_OFF;
  int* pref = (int*)(smem + SM::PREF_OFF);
  const uint32_t bar = sbase + SM::BAR_OFF;
  const uint32_t full_b = bar, empty_b = full_b + 8 * NPR;       // [NPR] ring entry landed / consumed
  const uint32_t rfull = empty_b + 8 * NPR, rempty = rfull + 16;  // [2] rotary block landed / consumed
  const uint32_t s_full = rempty + 16, s_free = s_full + 16;      // [2] scores complete / read
  const uint32_t p_full = s_free + 16, p_free = p_full + 16;      // [2] weights written / consumed (O^T holds the tile)
  const uint32_t o_free = p_free + 16;                            // [2] a set's O^T of an entry read out
  const uint32_t q_ready = o_free + 16;                           // the next entry's query is in shared memory
  const uint32_t fin_s = q_ready + 8, fin_o = fin_s + 8;
  const uint32_t red_b = fin_o + 8;                               // [2 sets][2] a tile's maxima posted
  const uint32_t post_b = red_b + 32;                             // [4 tiles] a tile's warps are done
  int4* tile_s = (int4*)(smem + SM::BAR_OFF + 384);   // [2]: {keys in the tile, boxes loaded, TILE_ bits, entry}
  volatile int* pv_fresh = (volatile int*)(smem + SM::BAR_OFF + 416);   // [2]: the set's first tile of an entry
  int4* start_s = (int4*)(smem + SM::BAR_OFF + 432);   // the first tile: {entry, its tile, its length}
  uint32_t* tmem_slot = (uint32_t*)(smem + SM::BAR_OFF + 480);
  volatile int* abort_word = (volatile int*)(smem + SM::BAR_OFF + 484);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x / a.groups, hg = blockIdx.x % a.groups;

  // ---- barriers (thread 64) and tensor memory (warp 1), beside the schedule (warp 0) ----
  if (threadIdx.x == 64) {
    for (int i = 0; i < NPR; ++i) { mbar_init(full_b + 8 * i, 1); mbar_init(empty_b + 8 * i, 1); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(rfull + 8 * i, 1);
      mbar_init(rempty + 8 * i, 5);   // read by the MMAs, and the scales by the set's warps
      mbar_init(s_full + 8 * i, 2);   // the MMAs, and the issuing thread (it has seen the query's scales)
      mbar_init(s_free + 8 * i, 4);
      mbar_init(p_full + 8 * i, 4);
      mbar_init(p_free + 8 * i, 1);
      mbar_init(o_free + 8 * i, 4);
    }
    for (int i = 0; i < 4; ++i) { mbar_init(red_b + 8 * i, 4); mbar_init(post_b + 8 * i, 4); }
    mbar_init(q_ready, 4);
    mbar_init(fin_s, 1);
    mbar_init(fin_o, 1);
    *abort_word = 0;
    fence_mbar_init();
  }
  griddep_wait();   // the inputs all come from the stream's earlier kernels, and those may still need their TMEM
  if (warp == 1) { tmem_alloc(smem_u32(tmem_slot), 512); tmem_relinquish(); }
  // ---- the schedule ----
  const int T_flat = a.flat ? (a.len + 127) / 128 : 0;
  if (!a.flat && warp == 0) {
    const int each = (a.n_ent + 31) / 32;   // n_ent <= A8_MAX_ENT
    int sum = 0;
    for (int k = 0; k < each; ++k) {
      const int e = each * lane + k;
      if (e >= a.n_ent) break;
      const int L = a8_len(a, e);
      if (blockIdx.x == 0 && (L == 0 && (a.min_ctx > 0 || a.ctx[e] != 0))) set_flag(a.flag, MLA_FLAG_BAD_CONTEXT);
      pref[e] = sum;
      sum += (L + 127) / 128;
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    // and the tile that this CTA begins with: one lane's entry holds it
    const int all = __shfl_sync(0xffffffffu, incl, 31), g = c * max(1, (all + a.units - 1) / a.units);
    for (int k = 0; k < each; ++k) {
      const int e = each * lane + k;
      if (e >= a.n_ent) break;
      const int b0 = pref[e] + incl - sum;
      pref[e] = b0;
      if (b0 <= g) {
        const int L = a8_len(a, e);
        if (g < b0 + (L + 127) / 128) *start_s = make_int4(e, g - b0, L, 0);
      }
    }
    if (lane == 31) pref[a.n_ent] = all;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (threadIdx.x == 0) griddep_launch_dependents();
  Walk8 w0{a.flat ? nullptr : pref, T_flat, a.n_ent, 0, 0, 0, 0};
  const int total = w0.at(a.n_ent);
  const int per = max(1, (total + a.units - 1) / a.units);
  if (blockIdx.x == 0)
    for (int e = threadIdx.x; e < a.n_ent; e += blockDim.x) {
      const int b0 = w0.at(e), b1 = w0.at(e + 1);
      a.seg[e] = b1 > b0 ? make_int2(b0 / per, (b1 - 1) / per - b0 / per + 1) : make_int2(0, 0);
    }
  const long long g0l = (long long)c * per;
  if (g0l >= total) {
    if (warp == 1) tmem_dealloc(tmem, 512);
    return;
  }
  const int g0 = (int)g0l, N = min(total - g0, per);
  if (a.flat) {
    w0.e = g0 / T_flat;
    w0.lt = g0 - w0.e * T_flat;
    w0.len = a.len;
  } else {
    const int4 at = *start_s;
    w0.e = at.x; w0.lt = at.y; w0.len = at.z;
  }
  w0.tiles = (w0.len + 127) / 128;

  if (warp == 8) {
    // ---------------- TMA: lane k < 128 / box brings rows [box k, box k + box) of each tile ----------------
    if (lane == 0) {
      prefetch_tmap(&tm_codes);
      prefetch_tmap(&tm_rope);
    }
    const int nb = 128 / a.box, none = max(a.n_blocks, 1);   // a block id beyond the map
    Walk8 w = w0;
    // this lane's box of the walk's tile, one tile ahead of its use: the block id as loaded (so that
    // nothing waits for it) and the first row within the block
    int raw = 0, off = 0;
    bool has = false;
    auto fetch_box = [&](const Walk8& v) {
      const int j = 128 * v.lt + a.box * lane;
      has = lane < nb && j < v.len;
      if (has) {
        const int at = j / a.bs;
        off = j - at * a.bs;
        raw = a.table[v.e * a.table_stride + at];
      }
    };
    fetch_box(w);
    int i = 0, odd = 0;
    bool ok = true, prev_first = false;
    for (; i < N; ++i) {
      const bool good = has && raw >= 0 && raw < a.n_blocks;
      if (has && !good && hg == 0) set_flag(a.flag, MLA_FLAG_BAD_BLOCK);
      const int cur = good ? raw : none, row0 = good ? off : 0;   // a block beyond the map: the load fills zeros
      const uint32_t boxes = __ballot_sync(0xffffffffu, good);
      const bool first = i == 0 || w.lt == 0;
      if (first && i > 0) odd ^= TILE_ODD;
      const int4 tile = make_int4(min(128, w.len - 128 * w.lt), (int)boxes,
                                  min(2, min(w.tiles - 1 - w.lt, N - 1 - i)) | (first ? TILE_FIRST : 0) |
                                      (prev_first ? TILE_PREV_FIRST : 0) | odd,
                                  w.e);
      prev_first = first;
      if (i + 1 < N) {
        w.next(a);
        fetch_box(w);
      }
      const uint32_t rb = rfull + 8 * (i & 1);
      if (!mbar_poll_warp(rempty + 8 * (i & 1), ((i >> 1) & 1) ^ 1, abort_word, a.flag)) { ok = false; break; }
      if (lane == 0) {
        tile_s[i & 1] = tile;
        mbar_arrive_expect_tx(rb, 16384 + __popc(boxes) * a.box * 4);
      }
      __syncwarp();
      if (lane < nb) tma_load_3d(rope_s + (i & 1) * 16384 + a.box * lane * 128, &tm_rope, rb, 0, row0, cur);
      if (good)
        bulk_load(sbase + SM::SC_OFF + (i & 1) * 512 + a.box * lane * 4,
                  a.cache + (long long)cur * a.block_bytes + a.sc_off + row0 * 4, a.box * 4, rb);
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int e = 2 * i + g, slot = e % NPR;
        if (!mbar_poll_warp(empty_b + 8 * slot, ((e / NPR) & 1) ^ 1, abort_word, a.flag)) { ok = false; break; }
        if (lane == 0) mbar_arrive_expect_tx(full_b + 8 * slot, 32768);
        __syncwarp();
        if (lane < nb)
          tma_load_5d(ring_s + slot * 32768 + (a.box * lane / 8) * 2048, &tm_codes, full_b + 8 * slot, 0, 0, 2 * g,
                      row0 / 8, cur);
      }
      if (!ok) break;
    }
    // drain what is in flight. When a wait gave up, tile i may lack some of its loads, and its
    // barriers are left alone: the earlier entries' phases have completed or will
    if (lane == 0 && i > 0) {
      for (int u = (2 * i > NPR ? 2 * i - NPR : 0); u < 2 * i; ++u) {
        const uint64_t t0 = global_timer_ns();
        while (!mbar_try_wait(full_b + 8 * (u % NPR), (u / NPR) & 1))
          if (global_timer_ns() - t0 > WAIT_LIMIT_NS) { set_flag(a.flag, MLA_FLAG_WAIT_TIMEOUT); break; }
      }
      for (int u = (i > 2 ? i - 2 : 0); u < i; ++u) {
        const uint64_t t0 = global_timer_ns();
        while (!mbar_try_wait(rfull + 8 * (u & 1), (u >> 1) & 1))
          if (global_timer_ns() - t0 > WAIT_LIMIT_NS) { set_flag(a.flag, MLA_FLAG_WAIT_TIMEOUT); break; }
      }
    }
    if (!ok && lane == 0) {   // loads of the unfinished tile: let them land before the CTA leaves
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 1000000ull) {}
    }
  } else if (warp == 8 + 1) {
    // ---------------- score MMAs (the whole warp runs the loop; see mma_f8_w) ----------------
    {
      constexpr uint32_t id_u = idesc_e4m3(128, 32), id_r = idesc_bf16(128, 16);
      const uint64_t d_ring = sdesc_sw128_sbo(ring_s, 2048), d_rope = sdesc_sw128(rope_s);
      const uint64_t d_q = sdesc_sw128(q_s), d_qpe = sdesc_sw128(qpe_s);
      int ks = 0;
      for (int i = 0; i < N; ++i) {
        const int b = i & 1;
        if (!mbar_poll_warp(rfull + 8 * b, (i >> 1) & 1, abort_word, a.flag) ||
            !mbar_poll_warp(s_free + 8 * b, ((i >> 1) & 1) ^ 1, abort_word, a.flag))
          break;
        if (tile_s[b].z & TILE_FIRST) {
          if (!mbar_poll_warp(q_ready, ks & 1, abort_word, a.flag)) break;
          ++ks;
        }
        tc_fence_after();
        const uint32_t d = tmem + SM::TM_S + 64 * b;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_bf16_w(d + 32, d_rope + (b * 16384 + 32 * k) / 16, d_qpe + 2 * k, id_r, k > 0 ? 1u : 0u);
        mma_commit_w(rempty + 8 * b);
        bool ok = true;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const int e = 2 * i + g, slot = e % NPR;
          if (!mbar_poll_warp(full_b + 8 * slot, (e / NPR) & 1, abort_word, a.flag)) { ok = false; break; }
          tc_fence_after();
          const uint64_t da = d_ring + (uint64_t)(slot * (32768 / 16));
#pragma unroll
          for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_f8_w(d, da + (kk * 1024 + 32 * k) / 16, d_q + ((2 * g + kk) * SM::QB + 32 * k) / 16, id_u,
                     (g > 0 || kk > 0 || k > 0) ? 1u : 0u);
        }
        if (!ok) break;
        mma_commit_w(s_full + 8 * b);
        if (lane == 0) mbar_arrive(s_full + 8 * b);
      }
      mma_commit_w(fin_s);
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(fin_s, 0))
        if (global_timer_ns() - t0 > WAIT_LIMIT_NS) { set_flag(a.flag, MLA_FLAG_WAIT_TIMEOUT); break; }
    }
  } else if (warp == 8 + 2) {
    // ---------------- value MMAs ----------------
    {
      constexpr uint32_t id_o = idesc_e4m3(128, 32, 1);
      // codes^T: one 128-column group along M, 8-key octets 2048 B apart along K
      const uint64_t d_v = sdesc_sw128_mn_sbo(ring_s, 1024, 2048), d_p = sdesc_sw128(p_s);
      int ko[2] = {0, 0};   // entries whose O^T the set has begun
      for (int i = 0; i < N; ++i) {
        const int b = i & 1;
        if (!mbar_poll_warp(p_full + 8 * b, (i >> 1) & 1, abort_word, a.flag)) break;
        const bool fresh = pv_fresh[b] != 0;
        if (fresh) {
          const int k = b ? ko[1]++ : ko[0]++;
          if (k > 0 && !mbar_poll_warp(o_free + 8 * b, (k - 1) & 1, abort_word, a.flag)) break;
        }
        tc_fence_after();
        const uint64_t dp = d_p + (uint64_t)(b * (SM::PB / 16));
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const int slot = (2 * i + g) % NPR;
          const uint64_t dv = d_v + (uint64_t)(slot * (32768 / 16));
#pragma unroll
          for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_f8_w(tmem + SM::TM_O + 128 * b + (2 * g + kk) * 32, dv + (kk * 1024 + 8192 * k) / 16, dp + 2 * k, id_o,
                     (!fresh || k > 0) ? 1u : 0u);
          mma_commit_w(empty_b + 8 * slot);
        }
        mma_commit_w(p_free + 8 * b);
      }
      mma_commit_w(fin_o);
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(fin_o, 0))
        if (global_timer_ns() - t0 > WAIT_LIMIT_NS) { set_flag(a.flag, MLA_FLAG_WAIT_TIMEOUT); break; }
    }
  } else {
    // ---------------- softmax: set b takes the tiles of parity b; thread <-> key of the tile ----------------
    const int set = warp >> 2, q = warp & 3;
    const int row = threadIdx.x & 127;
    const uint32_t lane_base = (uint32_t)(q * 32) << 16;
    float* red = (float*)(smem + SM::RED_OFF);                        // [2 sets][2][4][16]
    float* slq = red + SM::RED_SLQ;                                   // [2][16]: scale log2(e) 2^k_h
    float* rl = red + SM::RED_RL;                                     // [4][4][16]
    float* rp_s = red + SM::RED_RP;                                   // [4][16]
    float* ref_w = red + SM::RED_WARP + warp * 32;                    // [16] 8 - R, this warp's copy
    float* al_w = ref_w + 16;                                         // [16] factors of a rescale
    const uint32_t tm_o = tmem + SM::TM_O + lane_base;                // + 128 set + 32 group
    uint8_t* const pb = smem + SM::P_OFF + set * SM::PB + (row & 15);

    // The 16 heads' query rows of entry e in two E4M3 parts: eight threads per head, 64 columns each,
    // in two halves.
    auto load_q = [&](int e, int odd) {
      const int hd = row >> 3, sub = row & 7;
      const int r_hi = 16 * (hd >> 3) + (hd & 7);   // operand row of the first part; the second is 8 further on
      const long long r0 = a.flat ? (long long)e * 16 : (long long)e * a.H + 16LL * hg;
      const bool live = a.flat ? r0 + hd < a.rows_total : 16 * hg + hd < a.H;
      const uint4* src = reinterpret_cast<const uint4*>(a.q_abs + (live ? r0 + hd : 0) * 512 + 64 * sub);
      uint4 v[8];
      float m = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = live ? src[k] : make_uint4(0, 0, 0, 0);
      const uint4 pe = live ? reinterpret_cast<const uint4*>(a.q_pe + (r0 + hd) * 64)[sub] : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t u[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          m = fmaxf(m, fmaxf(finite_abs(__uint_as_float(u[j] << 16)), finite_abs(__uint_as_float(u[j] & 0xFFFF0000u))));
      }
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      // as a cache row's exponent, over bf16's whole range
      int k = 0;
      if (m > 0.f) {
        const uint32_t mb = __float_as_uint(m);
        k = (int)(mb >> 23) - 127 - ((mb & 0x7FFFFFu) > 0x600000u ? 7 : 8);
        k = max(-110, min(119, k));
      }
      const float inv = exp2_int(-k);
      if (sub == 0) slq[(odd ? 16 : 0) + hd] = a.scale_log2 * exp2_int(k);
      uint8_t* qb = smem + SM::Q_OFF + (sub >> 1) * SM::QB;   // columns [128 j, 128 j + 128) are k-block j
#pragma unroll
      for (int ch = 0; ch < 4; ++ch) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 vv = v[2 * ch + (j >> 1)];
          const uint32_t u0 = (j & 1) ? vv.z : vv.x, u1 = (j & 1) ? vv.w : vv.y;
          const float f0 = nan_if_inf(__uint_as_float(u0 << 16)) * inv, f1 = nan_if_inf(__uint_as_float(u0 & 0xFFFF0000u)) * inv;
          const float f2 = nan_if_inf(__uint_as_float(u1 << 16)) * inv, f3 = nan_if_inf(__uint_as_float(u1 & 0xFFFF0000u)) * inv;
          const uint16_t a0 = e4m3x2_sat(f0, f1), a1 = e4m3x2_sat(f2, f3);
          const float2 g0v = e4m3x2_f32(a0), g1v = e4m3x2_f32(a1);
          hi[j] = (uint32_t)a0 | ((uint32_t)a1 << 16);
          lo[j] = (uint32_t)e4m3x2_sat((f0 - g0v.x) * A8_QLO, (f1 - g0v.y) * A8_QLO) |
                  ((uint32_t)e4m3x2_sat((f2 - g1v.x) * A8_QLO, (f3 - g1v.y) * A8_QLO) << 16);
        }
        const int chunk = ((sub & 1) * 4 + ch) ^ (hd & 7);
        *reinterpret_cast<uint4*>(qb + r_hi * 128 + 16 * chunk) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(qb + (r_hi + 8) * 128 + 16 * chunk) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
      *reinterpret_cast<uint4*>(smem + SM::QPE_OFF + hd * 128 + 16 * (sub ^ (hd & 7))) = pe;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_ready);
    };

    const int box_log = 31 - __clz(a.box);
    const uint32_t all_boxes = (1u << (128 / a.box)) - 1u;
    // lane h < 16: head h's reference, the largest seen and the largest of late, over this set's tiles
    float R = -INFINITY, top = -INFINITY, recent = -INFINITY;
    float l[16];
#pragma unroll
    for (int h = 0; h < 16; ++h) l[h] = 0.f;
    bool ok = true;
    if (set == 0) load_q(w0.e, 0);   // while the first tile is on its way
    for (int i = set; i < N && ok; i += 2) {
      if (!mbar_poll_warp(rfull + 8 * set, (i >> 1) & 1, abort_word, a.flag)) { ok = false; break; }
      const int4 tile = tile_s[set];
      const bool first = tile.z & TILE_FIRST, prev_first = tile.z & TILE_PREV_FIRST;
      const int left = tile.z & TILE_LEFT;
      if (first && i > 0) {
        // the scores of the entry before are complete: its query may be replaced
        if (!mbar_poll_warp(s_full + 8 * (set ^ 1), ((i - 1) >> 1) & 1, abort_word, a.flag)) { ok = false; break; }
        load_q(tile.w, tile.z & TILE_ODD);
      }
      const float sj = *reinterpret_cast<const float*>(smem + SM::SC_OFF + set * 512 + row * 4);
      const bool valid = row < tile.x && (((uint32_t)tile.y >> (row >> box_log)) & 1u);
      // 2^k_j; rows never written (scale 0) count as zero rows
      const int kj = max(C8_KMIN, min(C8_KMAX, (int)(__float_as_uint(sj) >> 23) - 127));
      if (!mbar_poll_warp(s_full + 8 * set, (i >> 1) & 1, abort_word, a.flag)) { ok = false; break; }
      tc_fence_after();
      float y[16];
      {
        const float* sq = slq + (tile.z & TILE_ODD ? 16 : 0);
        const uint32_t sa = tmem + SM::TM_S + 64 * set + lane_base;
        uint32_t u[32], rp[16];
        tmem_ld16(sa, u);
        tmem_ld16(sa + 16, u + 16);
        tmem_ld16(sa + 32, rp);
        tmem_ld_wait<32>(u);
        tmem_ld_pin<16>(rp);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float4 s4 = *reinterpret_cast<const float4*>(sq + 4 * k);
          const float2 sv[2] = {make_float2(s4.x, s4.y), make_float2(s4.z, s4.w)};
          const float2 sj2 = make_float2(sj, sj), zero2 = make_float2(-0.f, -0.f);
#pragma unroll
          for (int j = 0; j < 4; j += 2) {
            const int h = 4 * k + j, at = 16 * (h >> 3) + (h & 7);
            auto pair = [](const uint32_t* x) { return make_float2(__uint_as_float(x[0]), __uint_as_float(x[1])); };
            const float2 uu = fma2(pair(u + at + 8), make_float2(1.f / A8_QLO, 1.f / A8_QLO), pair(u + at));
            const float2 rot = fma2(pair(rp + h), make_float2(a.scale_log2, a.scale_log2), make_float2((float)kj, (float)kj));
            const float2 yy = fma2(uu, fma2(sj2, sv[j >> 1], zero2), rot);
            y[h] = yy.x;
            y[h + 1] = yy.y;
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) { mbar_arrive(s_free + 8 * set); mbar_arrive(rempty + 8 * set); }
      }
      if (tile.x < 128 || (uint32_t)tile.y != all_boxes) {   // also drops NaN in rows that are no keys
#pragma unroll
        for (int h = 0; h < 16; ++h) y[h] = valid ? y[h] : -INFINITY;
      }
      // the tile's largest per head: within the warp here, over the set's four warps by lane h for head h
      const int slot = set * 2 + ((i >> 1) & 1);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float4 mx;
        mx.x = warp_max_f32(y[4 * k]);
        mx.y = warp_max_f32(y[4 * k + 1]);
        mx.z = warp_max_f32(y[4 * k + 2]);
        mx.w = warp_max_f32(y[4 * k + 3]);
        if (lane == 0) *reinterpret_cast<float4*>(red + (slot * 4 + q) * 16 + 4 * k) = mx;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(red_b + 8 * slot);
      // W(i - 2) has been consumed, and O^T of this set is at rest
      if (!mbar_poll_warp(p_free + 8 * set, ((i >> 1) & 1) ^ 1, abort_word, a.flag) ||
          !mbar_poll_warp(red_b + 8 * slot, (i >> 2) & 1, abort_word, a.flag)) {
        ok = false;
        break;
      }
      const bool fresh = first || prev_first;   // this set's first tile of the entry
      {
        // Move R up when a head's largest is above it, down when the largest of late (`recent` forgets an
        // octave a tile) is below R - 6; then to two to three octaves above, and with it the heads that
        // are about to move up; not below 2^-40 of the largest seen, where a tile no longer counts (and
        // 2^(old - new) stays far from overflow). The four warps decide alike.
        float m = -INFINITY;
        if (lane < 16) {
          const float* rr = red + slot * 64 + lane;
          m = fmaxf(fmaxf(rr[0], rr[16]), fmaxf(rr[32], rr[48]));
        }
        if (fresh) R = top = recent = -INFINITY;
        top = fmaxf(top, m);
        recent = fmaxf(recent - 1.f, m);
        const float want = fmaxf(ceilf(recent) + 2.f, top - 40.f);
        const bool move = recent > -INFINITY && (m > R || (recent < R - 6.f && want < R));
        if (__any_sync(0xffffffffu, move) || fresh) {
          float al = 1.f;
          if (move || m > R - 1.f) {
            if (R > -INFINITY) al = ex2_approx(R - want);
            R = want;
          }
          if (lane < 16) {
            ref_w[lane] = R == -INFINITY ? 8.f : 8.f - R;
            al_w[lane] = al;
          }
          __syncwarp();
          if (!fresh) {
            tc_fence_after();
#pragma unroll
            for (int o = 0; o < 2; ++o) {
              const float4 f0 = *reinterpret_cast<const float4*>(al_w + 8 * o), f1 = *reinterpret_cast<const float4*>(al_w + 8 * o + 4);
              const float f[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
#pragma unroll
              for (int h = 0; h < 8; ++h) l[8 * o + h] *= f[h];
              uint32_t v[64];
#pragma unroll
              for (int g = 0; g < 4; ++g) tmem_ld16(tm_o + 128 * set + 32 * g + 16 * o, v + 16 * g);
              tmem_ld_wait<64>(v);
#pragma unroll
              for (int h = 0; h < 64; ++h) v[h] = __float_as_uint(__uint_as_float(v[h]) * f[h & 7]);
#pragma unroll
              for (int g = 0; g < 4; ++g) tmem_st16(tm_o + 128 * set + 32 * g + 16 * o, v + 16 * g);
            }
            tmem_st_wait();
            tc_fence_before();
          }
        }
      }
      const float un = exp2_int(-kj);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 r4 = *reinterpret_cast<const float4*>(ref_w + 4 * k);
        const float rv[4] = {r4.x, r4.y, r4.z, r4.w};
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
          const int h = 4 * k + j;
          const float2 yr = add2(make_float2(y[h], y[h + 1]), make_float2(rv[j], rv[j + 1]));
          const float e0 = ex2_approx(yr.x), e1 = ex2_approx(yr.y);
          const float2 ll = fma2(make_float2(e0, e1), make_float2(un, un), make_float2(l[h], l[h + 1]));
          l[h] = ll.x;
          l[h + 1] = ll.y;
          const uint16_t c_hi = e4m3x2_sat(e0, e1);
          const float2 lo = fma2(make_float2(e0, e1), make_float2(A8_WLO, A8_WLO), e4m3x2_times(c_hi, -A8_WLO));
          const uint16_t c_lo = e4m3x2_sat(lo.x, lo.y);
          uint8_t* p0 = pb + (16 * (h >> 3) + (h & 7)) * 128 + (((row >> 4) ^ (h & 7)) << 4);
          uint8_t* p1 = pb + (16 * (h >> 3) + (h & 7) + 1) * 128 + (((row >> 4) ^ ((h & 7) + 1)) << 4);
          p0[0] = (uint8_t)c_hi;
          p1[0] = (uint8_t)(c_hi >> 8);
          p0[8 * 128] = (uint8_t)c_lo;
          p1[8 * 128] = (uint8_t)(c_lo >> 8);
        }
      }
      if (!valid) {
        // rows past the end may hold anything (even NaN codes); their weight is 0, but 0 * NaN is not
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          uint8_t* rp = smem + SM::RING_OFF + ((2 * i + (g >> 1)) % NPR) * 32768 + (row >> 3) * 2048 + (g & 1) * 1024 +
                        (row & 7) * 128;
#pragma unroll
          for (int k = 0; k < 8; ++k) *reinterpret_cast<uint4*>(rp + 16 * k) = make_uint4(0, 0, 0, 0);
        }
      }
      if (row == 0) pv_fresh[set] = fresh;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full + 8 * set);
      if (left <= 1) {   // the set's last tile of the entry: its row sums and references, for the end
#pragma unroll
        for (int h = 0; h < 16; ++h) {
          const float v = warp_sum(l[h]);
          if (lane == 0) rl[((i & 3) * 4 + q) * 16 + h] = v;
          l[h] = 0.f;
        }
        if (q == 0 && lane < 16) rp_s[(i & 3) * 16 + lane] = R;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(post_b + 8 * (i & 3));
      if (left > 0) continue;
      // The entry's last tile here: both sets' sums and O^T, brought to the larger of their references;
      // thread <-> latent column. (The other set is at most one tile ahead: the scores of its tile i + 3
      // wait for this set to have read those of tile i + 2.)
      if (!mbar_poll_warp(post_b + 8 * (i & 3), (i >> 2) & 1, abort_word, a.flag)) { ok = false; break; }
      if (!first && !mbar_poll_warp(post_b + 8 * ((i - 1) & 3), ((i - 1) >> 2) & 1, abort_word, a.flag)) { ok = false; break; }
      const long long unit = (long long)hg * (a.units + a.n_ent) + c + tile.w;
      const int live = (int)min(16LL, a.flat ? a.rows_total - 16LL * tile.w : (long long)a.H - 16 * hg);
      if (lane < 16) {
        const float Ro = first ? -INFINITY : rp_s[((i - 1) & 3) * 16 + lane], Rc = fmaxf(R, Ro);
        const float* ra = rl + (i & 3) * 64 + lane;
        const float* rb = rl + ((i - 1) & 3) * 64 + lane;
        const float sa = ra[0] + ra[16] + ra[32] + ra[48], sb = first ? 0.f : rb[0] + rb[16] + rb[32] + rb[48];
        // a set without a reference has no keys of any weight (a sum of zero), or NaN scores alone (a NaN sum)
        const float fa = R == -INFINITY ? sa : ex2_approx(R - Rc), fb = Ro == -INFINITY ? sb : ex2_approx(Ro - Rc);
        ref_w[lane] = fa;
        al_w[lane] = fb;
        if (q == 0 && lane < live)   // natural-log units; the weights carry the factor 2^8
          *reinterpret_cast<float2*>(a.part_ml + (unit * 16 + lane) * 2) =
              make_float2((Rc - 8.f) * 0.69314718055994531f, (fa != 0.f ? fa * sa : 0.f) + (fb != 0.f ? fb * sb : 0.f));
      }
      __syncwarp();
      if (!mbar_poll_warp(p_free + 8 * set, (i >> 1) & 1, abort_word, a.flag)) { ok = false; break; }
      if (!first && !mbar_poll_warp(p_free + 8 * (set ^ 1), ((i - 1) >> 1) & 1, abort_word, a.flag)) { ok = false; break; }
      tc_fence_after();
      float* po = a.part_o + unit * 16 * 512 + row;
#pragma unroll 1
      for (int g = 0; g < 4; ++g) {
        uint32_t o[32];
        float out[16];
        tmem_ld16(tm_o + 128 * set + 32 * g, o);
        tmem_ld16(tm_o + 128 * set + 32 * g + 16, o + 16);
        tmem_ld_wait<32>(o);
#pragma unroll
        for (int h = 0; h < 16; ++h)
          out[h] = fmaf(__uint_as_float(o[16 * (h >> 3) + 8 + (h & 7)]), 1.f / A8_WLO, __uint_as_float(o[16 * (h >> 3) + (h & 7)]));
        if (!first) {
          tmem_ld16(tm_o + 128 * (set ^ 1) + 32 * g, o);
          tmem_ld16(tm_o + 128 * (set ^ 1) + 32 * g + 16, o + 16);
          tmem_ld_wait<32>(o);
#pragma unroll
          for (int h = 0; h < 16; ++h) {
            const float fa = ref_w[h], fb = al_w[h];
            const float ob = fmaf(__uint_as_float(o[16 * (h >> 3) + 8 + (h & 7)]), 1.f / A8_WLO, __uint_as_float(o[16 * (h >> 3) + (h & 7)]));
            out[h] = (fa != 0.f ? fa * out[h] : 0.f) + (fb != 0.f ? fb * ob : 0.f);
          }
        }
#pragma unroll
        for (int h = 0; h < 16; ++h)
          if (h < live) po[h * 512 + 128 * g] = out[h];
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(o_free + 8 * set);
        if (!first) mbar_arrive(o_free + 8 * (set ^ 1));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace tc
}  // namespace mla
