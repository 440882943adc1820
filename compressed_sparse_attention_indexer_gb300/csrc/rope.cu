// Heads of new tokens on their way to the attention: the RMS norm of each
// query and key head, the rotation by the token's position, and the place
// where the head goes: a buffer (csa_qk_rope), or a row of a cache pool in the
// layer's type or as E4M3 codes with one fp32 scale per row and head
// (csa_kv_append; values go there as they are).
//   y = x * (sum_i x_i^2 / dim + eps)^(-1/2) * weight        (norm = 0: y = x)
//   (y_a, y_b) -> (y_a cos - y_b sin, y_a sin + y_b cos),  angle = pos * theta_i
// for the R / 2 pairs (a, b) of the rotated dims; all in fp32, rounded once.
//
// Angles.  theta_i / (2 pi) is held as a 64-bit fraction of a turn, so that
// pos * theta_i modulo a turn is one wrapping 64-bit product, exact for any
// 32-bit position but for the fraction's own rounding (theta's 53 bits:
// 2^-54 |pos theta| turns); an fp32 product would be off by whole degrees at
// positions beyond 2^17.  The fractions of base^(-2i/R) come with the launch.
//
// Memory bound: every element is read once and written once.  G lanes (a
// power of two up to a warp) hold a head as pairs of 8-element units, the two
// units that a rotation by halves pairs with one another in one lane, so that
// the rotation needs no exchange (kPaired); regions that do not fall on whole
// units take the partner's elements from memory a second time.
#include "csa_internal.cuh"
#include "ptx.cuh"
#include "rows.cuh"

namespace csa {

namespace {

constexpr int kThreads = 128;
constexpr int kUnit = 8;              // elements a lane loads together

struct Turns {
  uint64_t t[kRopeMaxDim / 2];        // theta_i / (2 pi) in units of 2^-64 turns
};

// theta / (2 pi) as a fraction of 2^-64 turns.
__device__ __forceinline__ uint64_t turn_of(float theta) {
  double t = (double)theta * 0.15915494309189535;
  t -= rint(t);
  return (uint64_t)(int64_t)(t * 18446744073709551616.0);
}

template <typename T>
struct Unit {
  static constexpr int V = kUnit / VecOf<T>::E;
  uint4 r[V];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < V; ++i) r[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void unpack(float* f) const {
#pragma unroll
    for (int i = 0; i < V; ++i) VecOf<T>::unpack(r[i], f + i * VecOf<T>::E);
  }
  static __device__ __forceinline__ void store(T* p, const float* f) {
#pragma unroll
    for (int i = 0; i < V; ++i) reinterpret_cast<uint4*>(p)[i] = VecOf<T>::pack(f + i * VecOf<T>::E);
  }
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// kTasks pairs of units per lane.  Tokens blockIdx.x * tb .. + tb - 1, their
// heads in order (queries, keys, values), nsub heads at a time.
template <typename T, int kTasks, bool kPaired, bool kFp8>
__global__ void __launch_bounds__(kThreads)
    heads_kernel(const HeadArgs a, const __grid_constant__ Turns turns, int lanes, int tb) {
  extern __shared__ float2 cs_sh[];                 // [tb][R / 2] (cos, sin)
  __shared__ int64_t row_sh[kThreads];              // pool row; -1: padding, -2: no such row
  __shared__ int pos_sh[kThreads];
  const int tid = threadIdx.x, sub = tid / lanes, nsub = kThreads / lanes, lane = tid % lanes;
  const int H = a.heads[0] + a.heads[1] + a.heads[2], half = a.R / 2;
  const int64_t first = (int64_t)blockIdx.x * tb;
  const int here = a.n - first < tb ? (int)(a.n - first) : tb;   // tokens of this block
  const int units = a.dim / kUnit, turned = kPaired ? a.R / (2 * kUnit) : 0, start = a.at / kUnit;
  pdl_wait();
  pdl_trigger();

  // the lane's units: paired ones first, then the rest in order
  int ua[kTasks][2];
#pragma unroll
  for (int i = 0; i < kTasks; ++i) {
    const int p = lane + i * lanes;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (p < turned) {
        ua[i][e] = start + p + e * turned;
      } else {
        const int x = (p - turned) * 2 + e, u = x < start || !kPaired ? x : x + 2 * turned;
        ua[i][e] = u < units ? u : -1;
      }
    }
  }
  // job: token `tok` of the block, head h of its H
  auto kind_of = [&](int h) { return h < a.heads[0] ? 0 : h < a.heads[0] + a.heads[1] ? 1 : 2; };
  auto head_in = [&](int h, int kind) { return kind == 0 ? h : kind == 1 ? h - a.heads[0] : h - a.heads[0] - a.heads[1]; };
  auto source = [&](int tok, int h) {
    const int kind = kind_of(h);
    return static_cast<const T*>(a.src[kind]) + (first + tok) * a.src_stride[kind] + head_in(h, kind) * a.dim;
  };
  Unit<T> next[kTasks][2];
  auto fetch = [&](int tok, int h) {
    if (tok >= here) return;
    const T* src = source(tok, h);
#pragma unroll
    for (int i = 0; i < kTasks; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (ua[i][e] >= 0) next[i][e].load(src + ua[i][e] * kUnit);
  };
  auto advance = [&](int& tok, int& h) {
    h += nsub;
    while (h >= H) h -= H, ++tok;
  };
  int tok = 0, h = sub;
  while (h >= H) h -= H, ++tok;
  fetch(tok, h);

  // ---- where the tokens go and their angles
  for (int x = tid; x < here; x += kThreads) {
    const int64_t t = first + x;
    int64_t row = t;
    int pos = 0;
    if (a.append) {
      int b = 0, s = 0;
      int64_t r = 0;
      bool pad = false, bad = false;
      if (a.ctx_len || a.count) b = (int)(t / a.S), s = (int)(t - (int64_t)b * a.S);
      int n = a.S;
      if (a.count) {
        n = a.count[b];
        bad = n < 0 || n > a.S;
        pad = bad || s >= n;
      }
      if (a.ctx_len) {
        const int len = a.ctx_len[b];
        bad |= len < 0;
        r = (int64_t)len - n + s;
        pad |= len < 0 || r < 0;
      }
      if (a.slot) {
        row = a.slot[t];
        pad |= row < 0;
      } else if (!pad) {
        row = -1;
        if (a.table) {
          const int64_t k = r / a.block;
          if (k < a.table_stride) {
            const int e = a.table[(int64_t)b * a.table_stride + k];
            if (e >= 0) row = (int64_t)e * a.block + (r - k * a.block);
          }
        } else {
          row = a.off[b] + r;
        }
      }
      if (!pad && (row < 0 || row >= a.rows)) row = -2, bad = true;
      if (pad) row = -1;
      if (bad && a.status) set_status(a.status, kStatusBadIndex);
      pos = (int)r;
    }
    if (a.pos) pos = a.pos[t];
    row_sh[x] = row;
    pos_sh[x] = pos;
  }
  __syncthreads();
  for (int x = tid; x < here * half; x += kThreads) {
    const int k = x / half, i = x - k * half;
    const uint64_t turn = a.freq ? turn_of(a.freq[i]) : turns.t[i];
    const uint64_t phase = turn * (uint64_t)(int64_t)pos_sh[k];
    float sn, cn;
    sincospif((float)(int)(phase >> 32) * 0x1p-31f, &sn, &cn);
    cs_sh[x] = make_float2(cn, sn);
  }
  __syncthreads();

  const float inv_dim = 1.f / (float)a.dim;
  const int steps = (here * H + nsub - 1) / nsub;   // the same for every thread (shuffles inside)
  for (int step = 0; step < steps; ++step) {
    const bool in = tok < here;
    float f[kTasks][2][kUnit];
#pragma unroll
    for (int i = 0; i < kTasks; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (in && ua[i][e] >= 0) {
          next[i][e].unpack(f[i][e]);
        } else {
#pragma unroll
          for (int x = 0; x < kUnit; ++x) f[i][e][x] = 0.f;
        }
      }
    const int tok0 = tok, h0 = h;
    advance(tok, h);
    fetch(tok, h);
    const int kind = kind_of(h0), head = head_in(h0, kind);
    const int64_t row = in ? row_sh[tok0] : -1;
    float r = 1.f;
    if (a.norm) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kTasks; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int x = 0; x < kUnit; ++x) sum = fmaf(f[i][e][x], f[i][e][x], sum);
      for (int o = lanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      r = rsqrtf(fmaf(sum, inv_dim, a.eps));
    }
    if (in && kind != 2) {
      const T* weight = static_cast<const T*>(a.weight[kind]);
      if (a.norm) {
#pragma unroll
        for (int i = 0; i < kTasks; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (ua[i][e] < 0) continue;
            float w[kUnit];
            if (weight) {
              Unit<T> u;
              u.load(weight + ua[i][e] * kUnit);
              u.unpack(w);
            }
#pragma unroll
            for (int x = 0; x < kUnit; ++x) f[i][e][x] *= weight ? r * w[x] : r;
          }
      }
      const float2* cs = cs_sh + tok0 * half;
      if constexpr (kPaired) {
#pragma unroll
        for (int i = 0; i < kTasks; ++i) {
          const int p = lane + i * lanes;
          if (p >= turned) continue;
          if (a.halves) {
#pragma unroll
            for (int x = 0; x < kUnit; ++x) {
              const float2 c = cs[p * kUnit + x];
              const float u = f[i][0][x], v = f[i][1][x];
              f[i][0][x] = u * c.x - v * c.y;
              f[i][1][x] = u * c.y + v * c.x;
            }
          } else {
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int x = 0; x < kUnit; x += 2) {
                const float2 c = cs[((p + e * turned) * kUnit + x) / 2];
                const float u = f[i][e][x], v = f[i][e][x + 1];
                f[i][e][x] = u * c.x - v * c.y;
                f[i][e][x + 1] = u * c.y + v * c.x;
              }
          }
        }
      } else if (half > 0) {
        const T* src = source(tok0, h0);
#pragma unroll
        for (int i = 0; i < kTasks; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int x = 0; x < kUnit; ++x) {
              const int d = ua[i][e] * kUnit + x - a.at;       // within the rotated dims
              if (ua[i][e] < 0 || d < 0 || d >= a.R) continue;
              const bool second = a.halves ? d >= half : d & 1;
              const int k = a.halves ? (second ? d - half : d) : d >> 1;
              const int other = a.at + (a.halves ? (second ? d - half : d + half) : d ^ 1);
              float o = to_f32(src[other]);
              if (a.norm) o *= weight ? r * to_f32(weight[other]) : r;
              const float2 c = cs[k];
              f[i][e][x] = second ? fmaf(f[i][e][x], c.x, o * c.y) : fmaf(f[i][e][x], c.x, -(o * c.y));
            }
      }
    }
    __syncwarp();   // a head's lanes have read what an output in place overwrites
    const bool quantised = kFp8 && kind != 0;
    float scale = 1.f;
    if (kFp8) {
      float most = 0.f;
#pragma unroll
      for (int i = 0; i < kTasks; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int x = 0; x < kUnit; ++x) most = fmaxf(most, fabsf(f[i][e][x]));
      for (int o = lanes / 2; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
      scale = block_scale(most);
    }
    if (row == -1 || (row < 0 && kind != 0)) continue;   // padding; no such row
    const int64_t to = kind == 0 || !a.append ? first + tok0 : row;
    if (quantised && lane == 0) a.scale[kind - 1][to * a.scale_stride + head] = scale;
#pragma unroll
    for (int i = 0; i < kTasks; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (ua[i][e] < 0) continue;
        const int64_t at = to * a.dst_stride[kind] + head * a.dim + ua[i][e] * kUnit;
        if (quantised) {
          divide<kUnit>(f[i][e], scale);
          uint32_t c[kUnit / 2];
#pragma unroll
          for (int x = 0; x < kUnit / 2; ++x)
            c[x] = __nv_cvt_float2_to_fp8x2(make_float2(f[i][e][2 * x], f[i][e][2 * x + 1]), __NV_SATFINITE, __NV_E4M3);
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.dst[kind]) + at) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
        } else {
          Unit<T>::store(static_cast<T*>(a.dst[kind]) + at, f[i][e]);
        }
      }
  }
}

template <typename T, int kTasks, bool kPaired>
int launch_shape(const HeadArgs& a, const Turns& turns, int lanes, int tb, bool fp8, cudaStream_t st, bool pdl) {
  const int64_t blocks = (a.n + tb - 1) / tb;
  const size_t smem = (size_t)tb * (a.R / 2) * sizeof(float2);
  return launch_kernel(fp8 ? heads_kernel<T, kTasks, kPaired, true> : heads_kernel<T, kTasks, kPaired, false>,
                       dim3((unsigned)blocks), dim3(kThreads), smem, st, pdl, a, turns, lanes, tb);
}

}  // namespace

int launch_heads(const HeadArgs& a, int dtype, bool fp8, double base, int num_sms, cudaStream_t st, bool pdl) {
  Turns turns;
  if (!a.freq && a.R > 0) {
    const double step = pow(base, -2.0 / a.R);
    double theta = 0.15915494309189535;   // 1 / (2 pi) of a turn per radian
    for (int i = 0; i < a.R / 2; ++i, theta *= step) turns.t[i] = (uint64_t)(theta * 18446744073709551616.0);
  }
  // whole units pair up where the rotated dims start on one and are a multiple of two
  const bool paired = a.at % kUnit == 0 && a.R % (2 * kUnit) == 0;
  const int units = a.dim / kUnit;
  const int tasks = paired ? a.R / (2 * kUnit) + (units - a.R / kUnit + 1) / 2 : (units + 1) / 2;
  int lanes = 1;
  while (lanes < tasks && lanes < 32) lanes *= 2;
  const int per = (tasks + lanes - 1) / lanes;   // 1, or 2 for heads of more than 64 units
  const int H = a.heads[0] + a.heads[1] + a.heads[2];
  // tokens per block: a few heads per lane, fewer where there are not enough tokens for the SMs
  const int nsub = kThreads / lanes;
  int64_t tb = (4 * nsub + H - 1) / H;
  const int64_t spread = (a.n + 4 * num_sms - 1) / (4 * num_sms);
  if (tb > spread) tb = spread;
  const int room = a.R > 0 ? 16384 / (a.R / 2 * (int)sizeof(float2)) : kThreads;
  if (tb > room) tb = room;
  if (tb > kThreads) tb = kThreads;
  while ((a.n + tb - 1) / tb > 0x7fffffff) ++tb;
#define CSA_HEADS(T)                                                                                          \
  (per == 1 ? paired ? launch_shape<T, 1, true>(a, turns, lanes, (int)tb, fp8, st, pdl)                       \
                     : launch_shape<T, 1, false>(a, turns, lanes, (int)tb, fp8, st, pdl)                      \
            : paired ? launch_shape<T, 2, true>(a, turns, lanes, (int)tb, fp8, st, pdl)                       \
                     : launch_shape<T, 2, false>(a, turns, lanes, (int)tb, fp8, st, pdl))
  return dtype == CSA_DTYPE_BF16 ? CSA_HEADS(__nv_bfloat16) : CSA_HEADS(float);
#undef CSA_HEADS
}

}  // namespace csa
