// The 8-bit latent cache: its block layout, the quantisation of a row, and the
// kernels that write rows into it and read them back (from a cache in the
// activation dtype too, where both are row copies).
//
// A block of `bs` rows holds three planes, so that a tile's codes, rotary keys
// and scales each are contiguous and 16-byte aligned for TMA:
//   [bs, r_kv] E4M3 codes | [bs, d_r] rotary keys (act dtype) | [bs] fp32 scales
// padded to a multiple of 128 bytes. Row j stands for
//   [scale_j * code_j | rotary_j]   (or the PE_FIRST order, when read back).
//
// One scale per row, a power of two 2^k with the least k that brings the row's
// largest finite magnitude to at most 448 (E4M3's largest), k in [-64, 7]:
//   - a power of two costs no accuracy in a floating-point code (it only shifts
//     the exponent) and makes scale * code exact in bf16 (4 significant bits),
//     so the cache read back is the cache attended to;
//   - one per row folds out of both products of the attention (it multiplies a
//     score, and a probability), so the tensor cores read the codes as they are.
// A latent row is RMS-normalised, so |c| <= sqrt(512) |gamma|; beyond 448 * 2^7
// = 57344 a value saturates. A value below 2^-10 of the code's unit (amax *
// 2^-18.8) rounds to zero. E4M3 has no infinity: NaN and infinities are stored
// as NaN, and the row's other values keep a scale of their own.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace mla {

struct Cache8 {
  int on;                 // 0: the cache holds act-dtype rows
  int bs, r_kv, d_r, esz; // esz: bytes of an act-dtype element (the rotary plane)
  long long pe_off, sc_off, block_bytes;
};

constexpr int C8_KMIN = -64, C8_KMAX = 7;

// k of a row whose largest finite magnitude is amax: 448 = 1.75 * 2^8, so
// amax = f * 2^e (1 <= f < 2) needs k = e - 8, or e - 7 when f > 1.75.
__device__ __forceinline__ int c8_exponent(float amax) {
  if (!(amax > 0.f)) return 0;
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 127;
  const int k = (b & 0x7FFFFFu) > 0x600000u ? e - 7 : e - 8;
  return k < C8_KMIN ? C8_KMIN : (k > C8_KMAX ? C8_KMAX : k);
}
__device__ __forceinline__ float exp2_int(int k) { return __uint_as_float((uint32_t)(k + 127) << 23); }   // |k| <= 126
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.4028234663852886e38f ? a : 0.f;   // NaN and infinities do not count
}
// Two E4M3 codes (round to nearest even, saturating), `lo` in the low byte;
// NaN and infinities become NaN.
__device__ __forceinline__ uint16_t e4m3x2_sat(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float nan_if_inf(float x) { return fabsf(x) == INFINITY ? __int_as_float(0x7fc00000) : x; }
__device__ __forceinline__ float2 e4m3x2_f32(uint16_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));   // exact: every E4M3 value is an f16
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Block-wide max of non-negative values (blockDim.x a multiple of 32). `red` >= 32 floats.
__device__ __forceinline__ float block_max_abs(float v, float* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  v = warp_max(v);
  __syncthreads();
  if (lane == 0) red[warp] = v;
  __syncthreads();
  return warp_max(lane < nw ? red[lane] : 0.f);
}

// Row `slot` of the 8-bit cache from one CTA: lat(i) the latent values as the
// act-dtype cache would hold them (in fp32), pe(i) the rotary values (TACT).
// Used by the front-fold kernels, which have the row in fp32 already.
template <typename TACT, typename LatFn>
__device__ __forceinline__ void c8_store_latent(const Cache8& c, uint8_t* cache, long long slot, LatFn lat, float* red) {
  float m = 0.f;
  for (int i = threadIdx.x; i < c.r_kv; i += blockDim.x) m = fmaxf(m, finite_abs(lat(i)));
  const int k = c8_exponent(block_max_abs(m, red));
  const float inv = exp2_int(-k);
  uint8_t* blk = cache + slot / c.bs * c.block_bytes;
  const long long r = slot % c.bs;
  uint16_t* codes = reinterpret_cast<uint16_t*>(blk + r * c.r_kv);   // r_kv is a multiple of 32
  for (int i = threadIdx.x; i < c.r_kv / 2; i += blockDim.x)
    codes[i] = e4m3x2_sat(nan_if_inf(lat(2 * i) * inv), nan_if_inf(lat(2 * i + 1) * inv));
  if (threadIdx.x == 0) reinterpret_cast<float*>(blk + c.sc_off)[r] = exp2_int(k);
}
template <typename TACT>
__device__ __forceinline__ TACT* c8_rotary(const Cache8& c, uint8_t* cache, long long slot) {
  return reinterpret_cast<TACT*>(cache + slot / c.bs * c.block_bytes + c.pe_off) + slot % c.bs * c.d_r;
}

// ---------------------------------------------------------------------------
// Rows in and out: a streaming copy, bound by HBM (1152 + 644 + 4 bytes a row for
// the DeepSeek latent in bf16). A warp takes four rows at a time, all their loads
// in flight before the first is used (one row at a time left half of the
// bandwidth idle: 68 us for 131007 rows written against 58, 41 us for 100003
// read against 33). Lane i takes the 8-element chunks i and i + 32 of the latent
// (r_kv <= 512) and chunk i of the rotary key, so that every load and store is a
// coalesced run of 8 or 16 bytes per lane.
// ---------------------------------------------------------------------------
struct CacheRowArgs {
  Cache8 c;
  void* rows;              // [n, r_kv + d_r] act dtype, in the order of `layout`
  uint8_t* cache;
  const int* slots;        // [n]; negative: the row is skipped
  long long n, n_rows;     // rows; cache rows (n_blocks * bs)
  int layout;
  int* flag;
};

template <typename T>
struct Chunk8 {            // eight elements as they lie in memory
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int j = 0; j < (int)sizeof(T) / 2; ++j) v[j] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void load(const void* p) {
#pragma unroll
    for (int j = 0; j < (int)sizeof(T) / 2; ++j) v[j] = reinterpret_cast<const uint4*>(p)[j];
  }
  __device__ __forceinline__ void store(void* p) const {
#pragma unroll
    for (int j = 0; j < (int)sizeof(T) / 2; ++j) reinterpret_cast<uint4*>(p)[j] = v[j];
  }
};
__device__ __forceinline__ void unpack8(const Chunk8<float>& c, float* f) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    f[4 * j] = __uint_as_float(c.v[j].x); f[4 * j + 1] = __uint_as_float(c.v[j].y);
    f[4 * j + 2] = __uint_as_float(c.v[j].z); f[4 * j + 3] = __uint_as_float(c.v[j].w);
  }
}
__device__ __forceinline__ void unpack8(const Chunk8<bf16>& c, float* f) {
  const uint32_t w[4] = {c.v[0].x, c.v[0].y, c.v[0].z, c.v[0].w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = __uint_as_float(w[j] << 16);
    f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void pack8(const float* f, Chunk8<float>* c) {
#pragma unroll
  for (int j = 0; j < 2; ++j)
    c->v[j] = make_uint4(__float_as_uint(f[4 * j]), __float_as_uint(f[4 * j + 1]), __float_as_uint(f[4 * j + 2]),
                         __float_as_uint(f[4 * j + 3]));
}
__device__ __forceinline__ void pack8(const float* f, Chunk8<bf16>* c) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
    w[j] = *reinterpret_cast<const uint32_t*>(&b);
  }
  c->v[0] = make_uint4(w[0], w[1], w[2], w[3]);
}

constexpr int CR_ROWS = 4;   // rows a warp has in flight

template <typename T, bool WRITE>
__global__ void __launch_bounds__(256) cache_rows_kernel(CacheRowArgs p) {
  griddep_wait();
  griddep_launch_dependents();
  const Cache8 c = p.c;
  const int lane = threadIdx.x & 31;
  const int R = c.r_kv + c.d_r, nch = c.r_kv / 8, npe = c.d_r / 8;
  const int lat_off = p.layout == MLA_ROW_LATENT_FIRST ? 0 : c.d_r;
  const int pe_off = p.layout == MLA_ROW_LATENT_FIRST ? c.r_kv : 0;
  const long long step = (long long)gridDim.x * 8 * CR_ROWS;
  for (long long t0 = (blockIdx.x * 8LL + (threadIdx.x >> 5)) * CR_ROWS; t0 < p.n; t0 += step) {
    int mine = -1;
    if (lane < CR_ROWS && t0 + lane < p.n) {
      mine = p.slots[t0 + lane];
      if (mine >= 0 && mine >= p.n_rows) {
        set_flag(p.flag, MLA_FLAG_BAD_SLOT);
        mine = -1;
      }
    }
    int slot[CR_ROWS];
#pragma unroll
    for (int k = 0; k < CR_ROWS; ++k) slot[k] = __shfl_sync(0xffffffffu, mine, k);
    if (!c.on) {   // an act-dtype cache: the rows as they are
      for (int i = lane; i < R / 8; i += 32) {
        Chunk8<T> v[CR_ROWS];
#pragma unroll
        for (int k = 0; k < CR_ROWS; ++k)
          if (slot[k] >= 0) v[k].load(WRITE ? (const T*)p.rows + (t0 + k) * R + 8 * i : (const T*)p.cache + (long long)slot[k] * R + 8 * i);
#pragma unroll
        for (int k = 0; k < CR_ROWS; ++k)
          if (slot[k] >= 0) v[k].store(WRITE ? (T*)p.cache + (long long)slot[k] * R + 8 * i : (T*)p.rows + (t0 + k) * R + 8 * i);
      }
      continue;
    }
    uint8_t* blk[CR_ROWS];
    int off[CR_ROWS];
#pragma unroll
    for (int k = 0; k < CR_ROWS; ++k) {
      const int b = slot[k] >= 0 ? slot[k] / c.bs : 0;
      off[k] = slot[k] >= 0 ? slot[k] - b * c.bs : 0;
      blk[k] = p.cache + b * c.block_bytes;
    }
    auto codes = [&](int k) { return reinterpret_cast<uint2*>(blk[k] + (long long)off[k] * c.r_kv); };
    auto rotary = [&](int k) { return reinterpret_cast<T*>(blk[k] + c.pe_off) + (long long)off[k] * c.d_r; };
    auto scale = [&](int k) { return reinterpret_cast<float*>(blk[k] + c.sc_off) + off[k]; };
    if (WRITE) {
      Chunk8<T> v[CR_ROWS][2], pe[CR_ROWS];
#pragma unroll
      for (int k = 0; k < CR_ROWS; ++k) {
        const T* row = (const T*)p.rows + (t0 + k) * R;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (slot[k] >= 0 && lane + 32 * h < nch) v[k][h].load(row + lat_off + 8 * (lane + 32 * h));
          else v[k][h].zero();
        }
        if (slot[k] >= 0 && lane < npe) pe[k].load(row + pe_off + 8 * lane);
      }
#pragma unroll
      for (int k = 0; k < CR_ROWS; ++k) {
        if (slot[k] < 0) continue;   // the same on every lane
        float m = 0.f;
        float f[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          unpack8(v[k][h], f);
#pragma unroll
          for (int j = 0; j < 8; ++j) m = fmaxf(m, finite_abs(f[j]));
        }
        const int e = c8_exponent(warp_max(m));
        const float inv = exp2_int(-e);
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (lane + 32 * h < nch) {
            unpack8(v[k][h], f);
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = e4m3x2_sat(nan_if_inf(f[2 * j] * inv), nan_if_inf(f[2 * j + 1] * inv));
            codes(k)[lane + 32 * h] = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
          }
        if (lane < npe) pe[k].store(rotary(k) + 8 * lane);
        for (int i = lane + 32; i < npe; i += 32) {
          Chunk8<T> x;
          x.load((const T*)p.rows + (t0 + k) * R + pe_off + 8 * i);
          x.store(rotary(k) + 8 * i);
        }
        if (lane == 0) *scale(k) = exp2_int(e);
      }
    } else {
      uint2 cc[CR_ROWS][2];
      float s[CR_ROWS];
      Chunk8<T> pe[CR_ROWS];
#pragma unroll
      for (int k = 0; k < CR_ROWS; ++k)
        if (slot[k] >= 0) {
          s[k] = *scale(k);
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (lane + 32 * h < nch) cc[k][h] = codes(k)[lane + 32 * h];
          if (lane < npe) pe[k].load(rotary(k) + 8 * lane);
        }
#pragma unroll
      for (int k = 0; k < CR_ROWS; ++k) {
        if (slot[k] < 0) continue;
        T* row = (T*)p.rows + (t0 + k) * R;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (lane + 32 * h < nch) {
            float f[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 x = e4m3x2_f32((uint16_t)((j < 2 ? cc[k][h].x : cc[k][h].y) >> (16 * (j & 1))));
              f[2 * j] = x.x * s[k];
              f[2 * j + 1] = x.y * s[k];
            }
            Chunk8<T> o;
            pack8(f, &o);
            o.store(row + lat_off + 8 * (lane + 32 * h));
          }
        if (lane < npe) pe[k].store(row + pe_off + 8 * lane);
        for (int i = lane + 32; i < npe; i += 32) {
          Chunk8<T> x;
          x.load(rotary(k) + 8 * i);
          x.store(row + pe_off + 8 * i);
        }
      }
    }
  }
}

}  // namespace mla
