// Latent attention over the paged cache in its general form: a 16/32-bit or an
// 8-bit cache (cache8.cuh), each sequence's own blocks and, optionally, a
// prefix that the whole batch shares, with o_lat and the log-sum-exp out.
//
//   s_hj = scale (q_abs_h . c_j + q_pe_h . k_pe_j)  over j in prefix, own rows
//   o_h  = sum_j softmax_j(s_h) c_j,   lse_h = log sum_j e^{s_hj}
//
// A softmax over a union of key sets is the (max, sum)-weighted mean of the
// softmaxes over its parts, so the prefix and the own rows run as passes of
// their own, each leaving split partials (unnormalised o, reference max m, sum
// l), and one kernel merges them. The prefix pass sees all n * H query rows
// against one set of keys: every prefix row is read from HBM once for the
// batch instead of once per sequence, and the rows fill the tensor core's
// tiles whatever H is.
#pragma once

#include "handle.cuh"
#include "simt_kernels.cuh"
#include "tc_attn8.cuh"
#include "tc_path.cuh"

namespace mla {

// Where a query row (token t, head h) finds its split partials.
struct MergeSrc {
  const float* o;       // [units, rows, r_kv]
  const float* ml;      // [units, rows, 2], and with half > 0 the same again ml_r floats further on
  const int2* seg;      // {first, count} of each entry: its units are first + entry ..; NULL: entry * splits ..
  const int* nseg;      // seg NULL: the partials in use of each entry's `splits` (NULL: all)
  long long ml_r;
  long long group_units;   // units of one group of `rows` heads (flat = 0)
  int half;             // columns c >= half use the second (m, l) copy (0: one copy)
  int splits, rows;
  int flat;             // entry = (t H + h) / rows; otherwise entry = e0 + t, and head group h / rows
  int e0;
  const float* corr;   // [units, rows] or NULL: the relative error of copy 0's sums (TcAttnArgs::corr)
};
struct MergeArgs {
  MergeSrc src[2];
  int n_src, H, r_kv;
  const float* sink;
  void* o;              // [n, H, r_kv]
  float* lse;           // [n, H] or NULL
  const int* ctx;       // a sequence whose length is invalid gets no keys at all
  int min_ctx, max_ctx;
  long long cap;
};

constexpr int MERGE_MAX = 640;   // split partials of one query row: at most one per SM and source

__device__ __forceinline__ long long merge_units(const MergeSrc& s, int H, int t, int h, int* count, int* row) {
  long long e, g = 0;
  if (s.flat) {
    const long long q = (long long)t * H + h;
    e = q / s.rows;
    *row = (int)(q % s.rows);
  } else {
    e = s.e0 + t;
    g = h / s.rows;
    *row = h % s.rows;
  }
  if (!s.seg) {
    *count = s.nseg ? min(s.nseg[e], s.splits) : s.splits;
    return g * s.group_units + e * s.splits;
  }
  const int2 f = s.seg[e];
  *count = f.y;
  return g * s.group_units + f.x + e;
}

// What brings copy 0's sum of weights p_j e^{d_j} back to the sum of p_j, for the log-sum-exp: corr = sum_j p_j d_j /
// sum_j p_j. e^{-corr} is that to first order, positive whatever the d_j (a partial score near f16's largest is
// rounded by more than one nat, which 1 - corr would make negative), and exact where one key holds the weight.
// Keys of weight zero with an infinite partial score leave a corr of NaN: the sum then stays as it is.
__device__ __forceinline__ float undo_corr(const float* corr, long long at) {
  const float c = corr ? corr[at] : 0.f;
  return c == c ? expf(-c) : 1.f;
}

// grid (n, H), 128 G threads: thread c % 128 owns four consecutive columns, the
// G groups of threads take every G-th partial and meet in shared memory (one
// token's 150 partials of 2 KB are a latency chain for a single group).
template <typename T>
__global__ void __launch_bounds__(1024) latent_merge_kernel(MergeArgs p) {
  __shared__ float wsh[2][MERGE_MAX];
  __shared__ float inv_sh[2];
  extern __shared__ float4 accs[];   // [G][128]
  const int t = blockIdx.x, h = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the lengths and the sink are older than the kernels that this one waits for
  const int L = p.ctx[t];
  const float z = p.sink ? p.sink[h] : -INFINITY;
  griddep_wait();
  griddep_launch_dependents();
  const bool live = L >= p.min_ctx && L <= p.max_ctx && (long long)L <= p.cap;
  int cnt0 = 0, cnt1 = 0, row0 = 0, row1 = 0;
  long long unit0 = merge_units(p.src[0], p.H, t, h, &cnt0, &row0), unit1 = 0;
  if (p.n_src > 1) unit1 = merge_units(p.src[1], p.H, t, h, &cnt1, &row1);
  if (!live) cnt0 = cnt1 = 0;
  cnt0 = min(cnt0, MERGE_MAX);
  const int total = min(cnt0 + cnt1, MERGE_MAX);
  // query row of partial i in its source's [units, rows] (source 1 from i = cnt0 on)
  auto at = [&](int i) {
    return i < cnt0 ? (unit0 + i) * p.src[0].rows + row0 : (unit1 + i - cnt0) * p.src[1].rows + row1;
  };
  const int c = (threadIdx.x & 127) * 4, grp = threadIdx.x >> 7, G = blockDim.x >> 7;
  auto part = [&](int i) {
    return *reinterpret_cast<const float4*>((i < cnt0 ? p.src[0].o : p.src[1].o) + at(i) * (long long)p.r_kv + c);
  };
  // the first partials are on their way while the weights are made
  constexpr int PRE = 4;
  float4 pre[PRE];
#pragma unroll
  for (int k = 0; k < PRE; ++k) {
    const int i = grp + k * G;
    pre[k] = c < p.r_kv && i < total ? part(i) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  if (warp < 2) {   // warp w: the weights from (m, l) copy w
    auto stats = [&](int i) {
      const MergeSrc& s = p.src[i < cnt0 ? 0 : 1];
      return *reinterpret_cast<const float2*>(s.ml + (warp && s.half ? s.ml_r : 0) + at(i) * 2);
    };
    float2 v0 = lane < total ? stats(lane) : make_float2(-INFINITY, 0.f);
    float M = v0.y > 0.f ? v0.x : -INFINITY;
    for (int i = lane + 32; i < total; i += 32) {
      const float2 v = stats(i);
      if (v.y > 0.f) M = fmaxf(M, v.x);
    }
    M = fmaxf(warp_max(M), z);
    float den = 0.f, den_l = 0.f;
    for (int i = lane; i < total; i += 32) {
      const float2 v = i == lane ? v0 : stats(i);
      const float w = v.y > 0.f ? __expf(v.x - M) : (v.y != v.y ? v.y : 0.f);   // a NaN sum stays NaN
      wsh[warp][i] = w;
      den += w == 0.f ? 0.f : w * v.y;
      if (warp == 0 && p.lse && w != 0.f) den_l += w * v.y * undo_corr(p.src[i < cnt0 ? 0 : 1].corr, at(i));
    }
    const float sink = z > -INFINITY ? __expf(z - M) : 0.f;
    den = warp_sum(den) + sink;
    den_l = warp_sum(den_l) + sink;
    if (lane == 0) {
      inv_sh[warp] = den == 0.f ? 0.f : 1.f / den;
      if (warp == 0 && p.lse) p.lse[(long long)t * p.H + h] = den == 0.f ? -INFINITY : M + logf(den_l);
    }
  }
  __syncthreads();
  // a source with one (m, l) copy is weighed by it for every column: both warps read the same one
  const int copy = (p.src[0].half && c >= p.src[0].half) || (p.n_src > 1 && p.src[1].half && c >= p.src[1].half);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float w, const float4& v) {
    if (w == 0.f) return;   // also where nothing was written
    acc.x = fmaf(w, v.x, acc.x); acc.y = fmaf(w, v.y, acc.y);
    acc.z = fmaf(w, v.z, acc.z); acc.w = fmaf(w, v.w, acc.w);
  };
  if (c < p.r_kv) {
#pragma unroll
    for (int k = 0; k < PRE; ++k)
      if (grp + k * G < total) add(wsh[copy][grp + k * G], pre[k]);
#pragma unroll 4
    for (int i = grp + PRE * G; i < total; i += G) add(wsh[copy][i], part(i));
  }
  if (G > 1) {
    accs[threadIdx.x] = acc;
    __syncthreads();
    if (grp == 0)
      for (int g = 1; g < G; ++g) {
        const float4 v = accs[128 * g + threadIdx.x];
        acc.x += v.x; acc.y += v.y; acc.z += v.z; acc.w += v.w;
      }
  }
  if (grp > 0 || c >= p.r_kv) return;
  const float inv = inv_sh[copy];
  T o[4] = {from_f32<T>(acc.x * inv), from_f32<T>(acc.y * inv), from_f32<T>(acc.z * inv), from_f32<T>(acc.w * inv)};
  T* dst = (T*)p.o + ((long long)t * p.H + h) * p.r_kv + c;   // a multiple of four elements from an output
  if (((uintptr_t)p.o & (4 * sizeof(T) - 1)) == 0) {           // that may lie anywhere
    if (sizeof(T) == 4) *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<uint4*>(o);
    else *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<uint2*>(o);
  } else {
    for (int k = 0; k < 4; ++k) dst[k] = o[k];
  }
}

}  // namespace mla

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// What one call attends to.
struct LatentCall {
  const void* q_abs; const void* q_pe; const void* cache;
  int n_blocks;
  const int32_t* prefix_table; int prefix_len;
  const int32_t* table; int mbps;
  const int32_t* ctx; int max_ctx;
  int n;
};

// Which kernels a call takes, how many tokens at a time, and where their partials lie.
struct LatentPlan {
  // The head-major launch takes the prefix, the own rows, or both; what it does not take runs on the
  // few-head 8-bit kernel, on mla_decode_attn's 16-bit kernels (own rows), or, all of it, on CUDA cores.
  bool heads_pre, heads_own, few_pre, few_own, own16, simt;
  int chunk;               // tokens per pass
  int splits;              // own16, simt: splits of the keys
  int units, groups;       // few_own: slices of the tile list, head groups
  int units_p, ents_p;     // few_pre: slices, entries
  int units_h, pre_h;      // head-major: SM pairs, prefix entries
  size_t o, ml, seg, o_h, ml_h, seg_h, total;   // own rows (or few_pre) apart; the head-major launch
  size_t o_p, ml_p, seg_p, corr_h;
};

constexpr int LAT_FEW_ROWS = 32;   // query rows up to which a prefix goes to the few-head 8-bit kernel
constexpr int LAT_MAX_HEADS = 128 * (ATT_MAX_SEQ - 1);

// `lse`: the log-sum-exp is wanted. `budget` > 0: the query is not 16-byte aligned, as the tensor-core kernels
// need it; CUDA cores then take as many tokens and splits at a time as this scratch holds. `force` < 0: by the
// rules; else bit 0 says whether a prefix goes to the head-major kernel and bit 1 whether the own rows ride
// along, as a smaller call may have it (latent_ws_bytes).
static inline LatentPlan latent_plan(const mla_handle* h, long long n, int prefix_len, int max_ctx, bool lse, size_t budget = 0,
                                     int force = -1) {
  const mla_config& c = h->cfg;
  const int H = c.n_heads;
  const int sms = h->tc.num_sms > 0 ? h->tc.num_sms : 148, pairs = sms / 2 > 0 ? sms / 2 : 1;
  LatentPlan w{};
  size_t off = 0;
  auto put = [&](size_t b) { size_t o = off; off = align_up(off + b, 256); return o; };
  // the tensor-core kernels: the DeepSeek latent, TMA boxes of whole parts of a block
  const bool tc = h->tc.attn && c.kv_lora_rank == 512 && c.qk_rope == 64;
  const bool b64 = c.block_size % 64 == 0, pre = prefix_len > 0;
  const long long tiles = cdiv(max_ctx, 64);
  // The own rows may ride in the prefix's head-major launch. With few heads that wastes most of its 128
  // rows (2 us per 64 rows and SM pair whatever the heads), but saves a launch with its start-up and tail
  // (about 17 us): worth it up to eight of such tiles per pair.
  const bool ride = H <= 128 && (force < 0 ? n * tiles <= 8LL * pairs : (force & 2) != 0);
  const bool fits = tc && (h->cache8 ? c.block_size % 16 == 0 : b64 && H <= 128);
  if (!fits || budget > 0) {
    w.simt = true;
  } else if (h->cache8) {
    // Per 128 keys the few-head kernel takes 2.2 us of one SM for every 16 heads (or 16 query rows), the
    // head-major one 4.1 us of two SMs whatever the rows up to 128. Own rows, 32 sequences of 8192:
    // 64 heads 111 against 126 us, 80 heads 139 against 128. A prefix of 16384: 48 rows 36 against 29 us,
    // since the head-major launch takes the own rows along.
    // (One token's query rows have to fit the head-major kernel's list of blocks of 128.)
    w.heads_pre = pre && b64 && H <= LAT_MAX_HEADS && (force < 0 ? n * H > LAT_FEW_ROWS : (force & 1) != 0);
    w.few_pre = pre && !w.heads_pre;
    w.heads_own = b64 && H <= 128 && (H > 64 || (w.heads_pre && ride));
    w.few_own = !w.heads_own;
  } else {
    // Beyond 32 heads only the head-major form of this file has the log-sum-exp good to fp32
    // (TcAttnArgs::corr); up to 32 the kernel of mla_decode_attn has a form for it. Own rows, with it and
    // without: 32 sequences of 4096 rows, 16 heads 46.4 and 45.4 us, 32 heads 70.9 with it; 64 sequences of
    // 1024 to 16384 rows, 128 heads 228 and 230.
    w.heads_pre = pre;
    w.heads_own = H > 32 ? pre || lse : pre && ride;
    w.own16 = !w.heads_own;
  }
  // tokens per pass: the kernels' entries (sequences; blocks of query rows) and tile lists
  long long most = n;
  auto limit = [&](long long m) { if (most > m) most = m > 0 ? m : 1; };
  if (w.simt) limit(65535);   // its grid
  if (w.few_own) limit(A8_MAX_ENT);
  if (w.own16 && H > 32) limit(ATT_MAX_SEQ);
  if (w.heads_pre || w.heads_own) {   // chunk + ceil(chunk H / 128) entries
    const long long per = (w.heads_own ? 128 : 0) + (w.heads_pre ? H : 0);
    limit((ATT_MAX_SEQ - 1) * 128LL / per);
  }
  if (!w.simt && force < 0) {   // tiles are counted in int
    const long long p = cdiv(prefix_len, 64) * cdiv(H, 16);
    limit((1 << 29) / (tiles > p ? tiles : p));
  }
  w.chunk = (int)most;
  if (w.few_own) {
    w.groups = (int)cdiv(H, 16);
    w.units = sms / w.groups > 0 ? sms / w.groups : 1;
    const size_t rows = (size_t)w.groups * (w.units + w.chunk) * 16;
    w.o = put(rows * 512 * 4);
    w.ml = put(rows * 2 * 4);
    w.seg = put((size_t)w.chunk * 8);
  } else if (!w.heads_own) {
    const long long s = cdiv((long long)(w.simt ? prefix_len : 0) + max_ctx, 256);
    w.splits = s < 2 ? 2 : (s > 16 ? 16 : (int)s);
    if (fits && budget > 0) {
      auto token = [&] { return (size_t)w.splits * H * (c.kv_lora_rank + 4) * 4; };
      const size_t most_bytes = budget > 768 ? budget - 768 : 0;   // less the roundings of `put`
      while (w.splits > 1 && token() > most_bytes) --w.splits;
      const size_t tokens = most_bytes / (token() + 4);
      if (tokens < (size_t)w.chunk) w.chunk = tokens > 0 ? (int)tokens : 1;
    }
    const size_t rows = (size_t)w.chunk * w.splits * H;
    w.o = put(rows * c.kv_lora_rank * 4);
    w.ml = put(rows * 2 * 4 * 2);   // one (m, l) copy per CTA of a pair
    w.seg = put((size_t)w.chunk * 4);
  }
  if (w.few_pre) {
    w.ents_p = (int)cdiv((long long)w.chunk * H, 16);
    w.units_p = sms;
    const size_t rows = (size_t)(w.units_p + w.ents_p) * 16;
    w.o_p = put(rows * 512 * 4);
    w.ml_p = put(rows * 2 * 4);
    w.seg_p = put((size_t)w.ents_p * 8);
  }
  if (w.heads_pre || w.heads_own) {
    w.units_h = pairs;
    w.pre_h = w.heads_pre ? (int)cdiv((long long)w.chunk * H, 128) : 0;
    const size_t ents = (size_t)w.pre_h + (w.heads_own ? w.chunk : 0), rows = (pairs + ents) * 128;
    w.o_h = put(rows * 512 * 4);
    w.ml_h = put(rows * 2 * 4 * 2);
    w.seg_h = put(ents * 8);
    w.corr_h = put(rows * 4);
  }
  w.total = off;
  return w;
}
// Enough for every call of up to these sizes: what a smaller one needs may be more where it takes other
// kernels. (An unaligned query makes do with what the aligned one has.)
static inline size_t latent_ws_bytes(const mla_handle* h, long long n, int prefix_len, int max_ctx) {
  size_t most = 0;
  const int H = h->cfg.n_heads, kinds = !h->cache8 && H > 32 ? 8 : 4;   // the log-sum-exp changes the plan there alone
  for (int p = 0; p < (prefix_len > 0 ? 2 : 1); ++p)
    for (int k = 0; k < kinds; ++k) {
      long long m = n;
      if (p && !(k & 1) && h->cache8 && h->cfg.block_size % 64 == 0 && H <= LAT_MAX_HEADS)
        m = n * H > LAT_FEW_ROWS ? LAT_FEW_ROWS / H : n;   // as many tokens as take a prefix to the few-head kernel
      const size_t t = m > 0 ? latent_plan(h, m, p ? prefix_len : 0, max_ctx, (k & 4) != 0, 0, k & 3).total : 0;
      if (t > most) most = t;
    }
  return most;
}

static inline void launch_merge(const MergeArgs& m, int n, int most, int o_dt, cudaStream_t s) {
  const int G = most <= 8 ? 1 : (most <= 24 ? 2 : (most <= 64 ? 4 : 8));
  const size_t smem = G > 1 ? (size_t)G * 128 * 16 : 0;
  const dim3 grid(n, m.H);
  if (o_dt == 0) launch_pdl(latent_merge_kernel<float>, grid, 128 * G, smem, s, m);
  else if (o_dt == 1) launch_pdl(latent_merge_kernel<bf16>, grid, 128 * G, smem, s, m);
  else launch_pdl(latent_merge_kernel<__half>, grid, 128 * G, smem, s, m);
  mla_count_launch(1);
}

// The 8-bit cache's planes as TMA sees them: the codes as {128 columns, 8 rows,
// 4 column groups, octets of a block, blocks}, boxes of two column groups and
// `box` rows; the rotary keys as {64, rows of a block, blocks}.
static int make_maps_cache8(CUtensorMap* codes, CUtensorMap* rope, const void* base, const Cache8& c, long long n_blocks,
                            int box) {
  auto fn = encode_fn();
  if (!fn) return MLA_ERR_CUDA;
  cuuint64_t d5[5] = {128, 8, 4, (cuuint64_t)(c.bs / 8), (cuuint64_t)n_blocks};
  cuuint64_t s5[4] = {512, 128, 4096, (cuuint64_t)c.block_bytes};
  cuuint32_t b5[5] = {128, 8, 2, (cuuint32_t)(box / 8), 1}, e5[5] = {1, 1, 1, 1, 1};
  CUresult r = fn(codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<void*>(base), d5, s5, b5, e5,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return MLA_ERR_CUDA;
  cuuint64_t d3[3] = {64, (cuuint64_t)c.bs, (cuuint64_t)n_blocks}, s3[2] = {128, (cuuint64_t)c.block_bytes};
  cuuint32_t b3[3] = {64, (cuuint32_t)box, 1}, e3[3] = {1, 1, 1};
  r = fn(rope, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, (char*)const_cast<void*>(base) + c.pe_off, d3, s3, b3, e3,
         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MLA_OK : MLA_ERR_CUDA;
}

static void launch_attn8(const CUtensorMap& codes, const CUtensorMap& rope, const TcAttn8Args& a, cudaStream_t s) {
  static std::atomic<bool> attr[64];
  set_smem_once(attr, tc_attn8_kernel, Attn8Smem::SIZE);
  launch_pdl(tc_attn8_kernel, (unsigned)(a.units * a.groups), A8_THREADS, Attn8Smem::SIZE, s, codes, rope, a);
  mla_count_launch(1);
}

// Largest part of a block that is a TMA box.
static int cache8_box(int bs) { return bs % 64 == 0 ? 64 : (bs % 32 == 0 ? 32 : 16); }

// A pass on the few-head 8-bit kernel: over the prefix (blocks of 16 query rows against its one
// table) or over each sequence's own rows.
static int pass_few8(const mla_handle* h, const LatentPlan& w, const LatentCall& a, bool pre, MergeArgs* m, char* scratch,
                     int* flag, cudaStream_t s) {
  const mla_config& c = h->cfg;
  const Cache8 c8 = cache8_of(h);
  const int box = cache8_box(c.block_size);
  CUtensorMap codes, rope;
  const int st = make_maps_cache8(&codes, &rope, a.cache, c8, a.n_blocks > 0 ? a.n_blocks : 1, box);
  if (st != MLA_OK) return st;
  TcAttn8Args k{};
  k.H = c.n_heads; k.rows_total = (long long)a.n * c.n_heads;
  k.mbps = a.mbps; k.bs = c.block_size; k.box = box; k.n_blocks = a.n_blocks;
  k.cache = (const uint8_t*)a.cache; k.block_bytes = c8.block_bytes; k.sc_off = c8.sc_off;
  k.q_abs = (const bf16*)a.q_abs; k.q_pe = (const bf16*)a.q_pe;
  k.scale_log2 = h->scale * 1.4426950408889634f;
  k.flag = flag;
  MergeSrc& q = m->src[m->n_src++];
  if (pre) {
    k.flat = 1; k.groups = 1; k.units = w.units_p;
    k.n_ent = (int)cdiv(k.rows_total, 16);
    k.len = a.prefix_len; k.table = a.prefix_table;
    k.part_o = (float*)(scratch + w.o_p); k.part_ml = (float*)(scratch + w.ml_p); k.seg = (int2*)(scratch + w.seg_p);
    q.flat = 1;
  } else {
    k.groups = w.groups; k.units = w.units; k.n_ent = a.n;
    k.ctx = a.ctx; k.min_ctx = m->min_ctx; k.max_ctx = a.max_ctx;
    k.table = a.table; k.table_stride = a.mbps;
    k.part_o = (float*)(scratch + w.o); k.part_ml = (float*)(scratch + w.ml); k.seg = (int2*)(scratch + w.seg);
    q.group_units = k.units + k.n_ent;
  }
  q.o = k.part_o; q.ml = k.part_ml; q.seg = k.seg; q.rows = 16;
  mla_timer_begin(pre ? "attn_prefix" : "attn", s);
  launch_attn8(codes, rope, k, s);
  mla_timer_end(pre ? "attn_prefix" : "attn", s);
  return MLA_OK;
}

template <bool C8, bool LSE>
static void launch_heads(const CUtensorMap& m0, const CUtensorMap& m1, const TcAttnArgs& k, const char* timer,
                         cudaStream_t s) {
  static std::atomic<bool> attr[64];
  set_smem_once(attr, tc_attn_decode_kernel<true, C8, LSE>, AttnSmemT<C8>::SIZE);
  mla_timer_begin(timer, s);
  launch_pdl(tc_attn_decode_kernel<true, C8, LSE>, 2 * k.units, C8 ? ATT_THREADS8 : ATT_THREADS, AttnSmemT<C8>::SIZE, s, m0, m1,
             k);
  mla_timer_end(timer, s);
  mla_count_launch(1);
}

// The head-major launch: the prefix (its 128 MMA rows take 128 query rows of any sequences), the own
// rows, or both, in one tile list.
static int pass_heads(const mla_handle* h, const LatentPlan& w, const LatentCall& a, MergeArgs* m, char* scratch, int* flag,
                      cudaStream_t s) {
  const mla_config& c = h->cfg;
  const int R = c.kv_lora_rank + c.qk_rope;
  const long long blocks = a.n_blocks > 0 ? a.n_blocks : 1;
  CUtensorMap mc, ml;
  int st;
  TcAttnArgs k{};
  if (h->cache8) {
    const Cache8 c8 = cache8_of(h);
    if ((st = make_maps_cache8(&ml, &mc, a.cache, c8, blocks, 64)) != MLA_OK) return st;
    k.c8 = (const uint8_t*)a.cache; k.c8_block = c8.block_bytes; k.c8_scales = c8.sc_off;
  } else {
    if ((st = make_map2(&mc, a.cache, R, blocks * c.block_size, R, 64)) != MLA_OK) return st;
    if ((st = make_map_cache_groups(&ml, a.cache, R, blocks * c.block_size, 4)) != MLA_OK) return st;
    k.lat_col0 = c.row_layout == MLA_ROW_LATENT_FIRST ? 0 : c.qk_rope;
    k.rope_col0 = c.row_layout == MLA_ROW_LATENT_FIRST ? c.kv_lora_rank : 0;
  }
  k.H = c.n_heads; k.rows_total = (long long)a.n * c.n_heads;
  k.n_pre = w.heads_pre ? (int)cdiv(k.rows_total, 128) : 0;
  k.n = k.n_pre + (w.heads_own ? a.n : 0);
  k.fixed_len = a.prefix_len; k.pre_table = a.prefix_table;
  k.block_table = a.table; k.mbps = a.mbps; k.ctx = a.ctx; k.max_ctx = a.max_ctx;
  k.allow_empty = m->min_ctx == 0;
  k.bs = c.block_size; k.n_blocks = a.n_blocks;
  k.q_abs = (const bf16*)a.q_abs; k.q_pe = (const bf16*)a.q_pe;
  k.scale_log2 = h->scale * 1.4426950408889634f;
  k.flag = flag; k.min_per = 1; k.units = w.units_h;
  k.part_o = (float*)(scratch + w.o_h); k.part_ml = (float*)(scratch + w.ml_h); k.seg = (int2*)(scratch + w.seg_h);
  k.ml_r = (long long)(k.units + k.n) * 128 * 2;
  k.corr = m->lse ? (float*)(scratch + w.corr_h) : nullptr;
  MergeSrc q{};
  q.corr = k.corr;
  q.o = k.part_o; q.ml = k.part_ml; q.ml_r = k.ml_r; q.half = 256; q.seg = k.seg; q.rows = 128;
  if (w.heads_pre) {
    q.flat = 1;
    m->src[m->n_src++] = q;
  }
  if (w.heads_own) {
    q.flat = 0;
    q.e0 = k.n_pre;
    m->src[m->n_src++] = q;
  }
  const char* timer = w.heads_pre ? "attn_prefix" : "attn";
  if (h->cache8) {
    if (k.corr) launch_heads<true, true>(mc, ml, k, timer, s);
    else launch_heads<true, false>(mc, ml, k, timer, s);
  } else {
    if (k.corr) launch_heads<false, true>(mc, ml, k, timer, s);
    else launch_heads<false, false>(mc, ml, k, timer, s);
  }
  return MLA_OK;
}

// The own rows of a 16-bit cache, as in mla_decode_attn.
static int pass_own16(const mla_handle* h, const LatentPlan& w, const LatentCall& a, MergeArgs* m, char* scratch,
                      int* flag, cudaStream_t s) {
  AttnParts P{};
  float* part_o = (float*)(scratch + w.o);
  float* part_ml = (float*)(scratch + w.ml);
  const int st = tc_attention_launch(h, a.q_abs, a.q_pe, a.cache, a.n_blocks, a.table, a.mbps, a.ctx, a.max_ctx, a.n,
                                     part_o, part_ml, w.splits, flag, (int*)(scratch + w.seg), a.prefix_len > 0, m->lse != nullptr, &P, s);
  if (st != MLA_OK) return st;
  MergeSrc& q = m->src[m->n_src++];
  q.o = part_o; q.ml = part_ml; q.ml_r = P.ml_r; q.half = P.half_cols; q.nseg = P.seg_counts; q.splits = P.splits;
  q.rows = h->cfg.n_heads;
  return MLA_OK;
}

// The same on CUDA cores (any shape, fp32 activations): the prefix rows simply
// come first in every sequence's list of keys.
static int pass_simt(const mla_handle* h, const LatentPlan& w, const LatentCall& a, MergeArgs* m, char* scratch, int* flag,
                     cudaStream_t s) {
  const mla_config& c = h->cfg;
  const int H = c.n_heads, rkv = c.kv_lora_rank, dr = c.qk_rope, R = rkv + dr;
  AttnArgs p{};
  p.q_abs = a.q_abs; p.q_pe = a.q_pe; p.cache = a.cache; p.n_blocks = a.n_blocks; p.bs = c.block_size;
  p.block_table = a.table; p.mbps = a.mbps; p.ctx = a.ctx; p.max_ctx = a.max_ctx;
  p.H = H; p.r_kv = rkv; p.d_r = dr; p.layout = c.row_layout; p.scale = h->scale;
  p.n_splits = w.splits;
  p.chunk = (int)(cdiv(cdiv((long long)a.prefix_len + a.max_ctx, w.splits), ATT_TR) * ATT_TR);
  p.part_o = (float*)(scratch + w.o); p.part_ml = (float*)(scratch + w.ml); p.flag = flag;
  p.prefix_table = a.prefix_table; p.prefix_len = a.prefix_len; p.c8 = cache8_of(h);
  const size_t smem = (size_t)(ATT_TR * (R + 1) + ATT_HPB * R) * 4;
  const dim3 grid(w.splits, a.n, (unsigned)cdiv(H, ATT_HPB));
  mla_timer_begin("attn", s);
  if (c.act_dtype == MLA_F32) {
    cudaFuncSetAttribute(attn_decode_simt_kernel<float, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    attn_decode_simt_kernel<float, true><<<grid, 256, smem, s>>>(p);
  } else {
    cudaFuncSetAttribute(attn_decode_simt_kernel<bf16, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    attn_decode_simt_kernel<bf16, true><<<grid, 256, smem, s>>>(p);
  }
  mla_timer_end("attn", s);
  mla_count_launch(1);
  MergeSrc& q = m->src[m->n_src++];
  q.o = p.part_o; q.ml = p.part_ml; q.splits = w.splits; q.rows = H;
  return MLA_OK;
}

// o_lat [n, H, r_kv] (o_dt: 0 fp32, 1 bf16, 2 f16) and, if given, lse [n, H]. `scratch`: bytes of them, at least
// latent_ws_bytes of the call's sizes.
static inline int latent_core(const mla_handle* h, const LatentCall& call, void* o_lat, int o_dt, float* lse, char* scratch,
                              size_t bytes, int* flag, cudaStream_t s) {
  const mla_config& c = h->cfg;
  const int H = c.n_heads, rkv = c.kv_lora_rank, dr = c.qk_rope;
  const size_t esz = c.act_dtype == MLA_F32 ? 4 : 2, o_esz = o_dt == 0 ? 4 : 2;
  const bool aligned = (((uintptr_t)call.q_abs | (uintptr_t)call.q_pe) & 15) == 0;
  const LatentPlan w = latent_plan(h, call.n, call.prefix_len, call.max_ctx, lse != nullptr, aligned ? 0 : bytes);
  for (int t = 0; t < call.n; t += w.chunk) {
    LatentCall a = call;
    a.n = call.n - t < w.chunk ? call.n - t : w.chunk;
    a.q_abs = (const char*)call.q_abs + (size_t)t * H * rkv * esz;
    a.q_pe = (const char*)call.q_pe + (size_t)t * H * dr * esz;
    a.table = call.table + (size_t)t * call.mbps;
    a.ctx = call.ctx + t;
    MergeArgs m{};
    m.H = H; m.r_kv = rkv;
    m.sink = h->has_sink ? (const float*)(h->base + h->L.sink) : nullptr;
    m.o = (char*)o_lat + (size_t)t * H * rkv * o_esz;
    m.lse = lse ? lse + (size_t)t * H : nullptr;
    m.ctx = a.ctx; m.min_ctx = a.prefix_len > 0 ? 0 : 1; m.max_ctx = a.max_ctx;
    m.cap = (long long)a.mbps * c.block_size;
    int st = MLA_OK;
    if (w.heads_pre || w.heads_own) st = pass_heads(h, w, a, &m, scratch, flag, s);
    if (st == MLA_OK && w.few_pre) st = pass_few8(h, w, a, true, &m, scratch, flag, s);
    if (st == MLA_OK && w.few_own) st = pass_few8(h, w, a, false, &m, scratch, flag, s);
    if (st == MLA_OK && w.own16) st = pass_own16(h, w, a, &m, scratch, flag, s);
    if (st == MLA_OK && w.simt) st = pass_simt(h, w, a, &m, scratch, flag, s);
    if (st != MLA_OK) return st;
    // split partials of one query row, about: each part's slices per entry, at most one per tile
    auto parts = [](long long slices, long long ents, long long tiles) {
      const long long k = cdiv(slices, ents > 0 ? ents : 1) + 1;
      return k < tiles ? k : tiles;
    };
    const long long t_own = cdiv(a.max_ctx, 64), t_pre = cdiv(a.prefix_len, 64);
    const long long ents_h = w.pre_h + (w.heads_own ? a.n : 0);
    long long most = w.splits;
    if (w.few_own) most += parts(w.units, a.n, t_own);
    if (w.few_pre) most += parts(w.units_p, w.ents_p, t_pre);
    if (w.heads_own) most += parts(w.units_h, ents_h, t_own);
    if (w.heads_pre) most += parts(w.units_h, w.heads_own && t_pre > 4 * t_own ? w.pre_h : ents_h, t_pre);
    launch_merge(m, a.n, (int)most, o_dt, s);
  }
  return MLA_OK;
}
