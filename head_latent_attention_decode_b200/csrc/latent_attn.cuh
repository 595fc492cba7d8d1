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
#include "tc_path.cuh"

namespace mla {

// Where a query row (token t, head h) finds its split partials.
struct MergeSrc {
  const float* o;       // [units, rows, r_kv]
  const float* ml;      // [units, rows, 2], and with half > 0 the same again ml_r floats further on
  const int2* seg;      // {first, count} of each entry: its units are first + entry ..; NULL: entry * splits ..
  long long ml_r;
  long long group_units;   // units of one group of `rows` heads (flat = 0)
  int half;             // columns c >= half use the second (m, l) copy (0: one copy)
  int splits, rows;
  int flat;             // entry = (t H + h) / rows; otherwise entry = t, and head group h / rows
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
    e = t;
    g = h / s.rows;
    *row = h % s.rows;
  }
  if (!s.seg) {
    *count = s.splits;
    return g * s.group_units + e * s.splits;
  }
  const int2 f = s.seg[e];
  *count = f.y;
  return g * s.group_units + f.x + e;
}

// grid (n, H), 128 G threads: thread c % 128 owns four consecutive columns, the
// G groups of threads take every G-th partial and meet in shared memory (one
// token's 150 partials of 2 KB are a latency chain for a single group).
template <typename T>
__global__ void __launch_bounds__(1024) latent_merge_kernel(MergeArgs p) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ float wsh[2][MERGE_MAX];
  __shared__ float inv_sh[2];
  extern __shared__ float4 accs[];   // [G][128]
  const int t = blockIdx.x, h = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int L = p.ctx[t];
  const bool live = L >= p.min_ctx && L <= p.max_ctx && (long long)L <= p.cap;
  int cnt[2] = {0, 0}, row[2] = {0, 0};
  long long unit[2] = {0, 0};
  for (int k = 0; k < p.n_src; ++k) unit[k] = merge_units(p.src[k], p.H, t, h, &cnt[k], &row[k]);
  if (!live) cnt[0] = cnt[1] = 0;
  cnt[0] = min(cnt[0], MERGE_MAX);
  const int total = min(cnt[0] + cnt[1], MERGE_MAX);
  if (warp < 2) {   // warp w: the weights from (m, l) copy w
    float M = -INFINITY;
    for (int i = lane; i < total; i += 32) {
      const int k = i >= cnt[0];
      const MergeSrc& s = p.src[k];
      const float* ml = s.ml + (warp && s.half ? s.ml_r : 0) + ((unit[k] + i - (k ? cnt[0] : 0)) * s.rows + row[k]) * 2;
      const float2 v = *reinterpret_cast<const float2*>(ml);
      if (v.y > 0.f || v.y != v.y) M = fmaxf(M, v.x);
    }
    M = warp_max(M);
    const float z = p.sink ? p.sink[h] : -INFINITY;
    M = fmaxf(M, z);
    float den = 0.f;
    for (int i = lane; i < total; i += 32) {
      const int k = i >= cnt[0];
      const MergeSrc& s = p.src[k];
      const float* ml = s.ml + (warp && s.half ? s.ml_r : 0) + ((unit[k] + i - (k ? cnt[0] : 0)) * s.rows + row[k]) * 2;
      const float2 v = *reinterpret_cast<const float2*>(ml);
      const float w = (v.y > 0.f) ? __expf(v.x - M) : (v.y != v.y ? v.y : 0.f);   // a NaN sum stays NaN
      wsh[warp][i] = w;
      den += w == 0.f ? 0.f : w * v.y;
    }
    den = warp_sum(den) + (z > -INFINITY ? __expf(z - M) : 0.f);
    if (lane == 0) {
      inv_sh[warp] = den == 0.f ? 0.f : 1.f / den;
      if (warp == 0 && p.lse) p.lse[(long long)t * p.H + h] = den == 0.f ? -INFINITY : M + logf(den);
    }
  }
  __syncthreads();
  const int c = (threadIdx.x & 127) * 4, grp = threadIdx.x >> 7, G = blockDim.x >> 7;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c < p.r_kv) {
#pragma unroll 4
    for (int i = grp; i < total; i += G) {
      const int k = i >= cnt[0];
      const MergeSrc& s = p.src[k];
      const float w = wsh[s.half && c >= s.half ? 1 : 0][i];
      if (w == 0.f) continue;
      const float4 v = *reinterpret_cast<const float4*>(
          s.o + ((unit[k] + i - (k ? cnt[0] : 0)) * s.rows + row[k]) * (long long)p.r_kv + c);
      acc.x = fmaf(w, v.x, acc.x); acc.y = fmaf(w, v.y, acc.y);
      acc.z = fmaf(w, v.z, acc.z); acc.w = fmaf(w, v.w, acc.w);
    }
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
  // the two copies differ only where a source has two; both cover every source
  const float inv = inv_sh[(p.src[0].half && c >= p.src[0].half) || (p.n_src > 1 && p.src[1].half && c >= p.src[1].half)];
  T* o = (T*)p.o + ((long long)t * p.H + h) * p.r_kv + c;
  o[0] = from_f32<T>(acc.x * inv); o[1] = from_f32<T>(acc.y * inv);
  o[2] = from_f32<T>(acc.z * inv); o[3] = from_f32<T>(acc.w * inv);
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

struct LatentWs {
  size_t o, ml, total;
  int splits;
};

static inline LatentWs latent_ws(const mla_handle* h, long long n, int prefix_len, int max_ctx) {
  LatentWs w{};
  const long long keys = (long long)prefix_len + max_ctx;
  const long long c = cdiv(keys, 256);
  w.splits = c < 2 ? 2 : (c > 16 ? 16 : (int)c);
  size_t off = 0;
  auto put = [&](size_t b) { size_t o = off; off = align_up(off + b, 256); return o; };
  const long long rows = n * w.splits * h->cfg.n_heads;
  w.o = put((size_t)rows * h->cfg.kv_lora_rank * 4);
  w.ml = put((size_t)rows * 2 * 4);
  w.total = off;
  return w;
}
static inline size_t latent_ws_bytes(const mla_handle* h, long long n, int prefix_len, int max_ctx) {
  return latent_ws(h, n, prefix_len, max_ctx).total;
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

// o_lat [n, H, r_kv] (o_dt: 0 fp32, 1 bf16, 2 f16) and, if given, lse [n, H].
static inline int latent_core(const mla_handle* h, const LatentCall& a, void* o_lat, int o_dt, float* lse, char* scratch,
                              int* flag, cudaStream_t s) {
  const mla_config& c = h->cfg;
  const int H = c.n_heads, rkv = c.kv_lora_rank, dr = c.qk_rope, R = rkv + dr;
  const LatentWs W = latent_ws(h, a.n, a.prefix_len, a.max_ctx);
  MergeArgs m{};
  m.H = H; m.r_kv = rkv;
  m.sink = h->has_sink ? (const float*)(h->base + h->L.sink) : nullptr;
  m.o = o_lat; m.lse = lse;
  m.ctx = a.ctx; m.min_ctx = a.prefix_len > 0 ? 0 : 1; m.max_ctx = a.max_ctx;
  m.cap = (long long)a.mbps * c.block_size;
  AttnArgs p{};
  p.q_abs = a.q_abs; p.q_pe = a.q_pe; p.cache = a.cache; p.n_blocks = a.n_blocks; p.bs = c.block_size;
  p.block_table = a.table; p.mbps = a.mbps; p.ctx = a.ctx; p.max_ctx = a.max_ctx;
  p.H = H; p.r_kv = rkv; p.d_r = dr; p.layout = c.row_layout; p.scale = h->scale;
  p.n_splits = W.splits;
  p.chunk = (int)(cdiv(cdiv((long long)a.prefix_len + a.max_ctx, W.splits), ATT_TR) * ATT_TR);
  p.part_o = (float*)(scratch + W.o); p.part_ml = (float*)(scratch + W.ml); p.flag = flag;
  p.prefix_table = a.prefix_table; p.prefix_len = a.prefix_len; p.c8 = cache8_of(h);
  const size_t smem = (size_t)(ATT_TR * (R + 1) + ATT_HPB * R) * 4;
  const dim3 grid(W.splits, a.n, (unsigned)cdiv(H, ATT_HPB));
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
  MergeSrc& q = m.src[0];
  q.o = p.part_o; q.ml = p.part_ml; q.splits = W.splits; q.rows = H;
  m.n_src = 1;
  launch_merge(m, a.n, W.splits, o_dt, s);
  return MLA_OK;
}
