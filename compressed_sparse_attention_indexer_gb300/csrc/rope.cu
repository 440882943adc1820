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
// 32-bit position but for the fraction's own rounding (theta's 53 bits, up to 16
// products and base's logarithm: 2^-46 |pos theta| at most); an fp32 product would be
// off by whole degrees at positions beyond 2^17.  The fractions of base^(-2i/R) come
// with the launch.
//
// Memory bound: every element is read once and written once.  G lanes (a
// power of two up to a warp) hold a head as pairs of 8-element units, the two
// units that a rotation by halves pairs with one another in one lane, so that
// the rotation needs no exchange (kPaired); regions that do not fall on whole
// units exchange their elements through shared memory.
//
// Measured: 16384 tokens of 32 + 8 heads of 128, bf16, 59 us (5.66 TB/s; with their
// values and into pages 70 us, 5.74 TB/s); 64 tokens of 65 heads of 576, 4.5 us; one
// token 3.5 .. 3.9 us, which is a launch.  131072 keys of 128 (64 dims turned) to E4M3 in 23 us
// (2.2 TB/s): 19 with 16 dims turned, 21 without the norm, 19 into a bf16 pool.  Regions off
// whole units: 16384 tokens as above with 24 dims turned 131 us (2.6 TB/s).
#include "csa_internal.cuh"
#include "ptx.cuh"
#include "rows.cuh"

namespace csa {

namespace {

constexpr int kThreads = 128;
constexpr int kUnit = 8;              // elements a lane loads together
constexpr int kJobs = 8;              // heads per lane of a block, where there are enough

struct Turns {
  uint64_t t[kRopeMaxDim / 2];        // theta_i / (2 pi) in units of 2^-64 turns
};

// How the blocks share the work: kind k's start at block start[k]; a block has tb[k] tokens
// and per[k] of their heads, one of splits[k] parts.
struct Plan {
  int start[4];
  int tb[3], splits[3], per[3];
};

// theta / (2 pi) as a fraction of 2^-64 turns.
__device__ __forceinline__ uint64_t turn_of(float theta) {
  double t = (double)theta * 0.15915494309189535;
  t -= rint(t);
  return (uint64_t)(int64_t)(t * 18446744073709551616.0);
}

// Cosine and sine of phase 2^-32 turns: the quarter turn nearest, and the rest of at most an
// eighth (|x| <= pi / 4) by the Taylor series of either, cut off below 2e-9: off by less
// than 2.5 2^-24 with the rounding of x to fp32.
__device__ __forceinline__ void cos_sin(uint32_t phase, float& cn, float& sn) {
  const uint32_t quarter = (phase + 0x20000000u) >> 30;
  const float x = (float)(int)(phase - (quarter << 30)) * 1.4629180792671596e-9f;   // 2 pi / 2^32
  const float y = x * x;
  const float s = fmaf(x * y, fmaf(y, fmaf(y, fmaf(y, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f), x);
  const float c = fmaf(y, fmaf(y, fmaf(y, fmaf(y, fmaf(y, -1.f / 3628800.f, 1.f / 40320.f), -1.f / 720.f), 1.f / 24.f), -0.5f), 1.f);
  const float a = quarter & 1 ? s : c, b = quarter & 1 ? c : s;
  cn = __uint_as_float(__float_as_uint(a) ^ ((quarter + 1) & 2) << 30);
  sn = __uint_as_float(__float_as_uint(b) ^ (quarter & 2) << 30);
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

// Two fp32 products in one instruction.
__device__ __forceinline__ void mul2(float* d, float b0, float b1) {
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %3};\n mul.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}\n"
      : "+f"(d[0]), "+f"(d[1])
      : "f"(b0), "f"(b1));
}
__device__ __forceinline__ void fma2(float* d, const float* a, const float* b) {   // d += a b
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %3};\n mov.b64 z, {%4, %5};\n fma.rn.f32x2 x, y, z, x;\n"
      " mov.b64 {%0, %1}, x;\n}\n"
      : "+f"(d[0]), "+f"(d[1])
      : "f"(a[0]), "f"(a[1]), "f"(b[0]), "f"(b[1]));
}

// A block does heads of one kind (queries, keys or values) of some tokens (see Plan),
// nsub heads at a time, kTasks pairs of units per lane.  The kind is the block's, so
// that its norm, rotation and destination are branches of the whole block and the weight
// stays in registers.  (All kinds in one block, one after the other: 64 x 65 heads of
// 576 dims in 13 us instead of 5.)
template <typename T, int kTasks, bool kPaired, bool kFp8>
__global__ void __launch_bounds__(kThreads)
    heads_kernel(const HeadArgs a, const __grid_constant__ Turns turns, const __grid_constant__ Plan plan, int lanes) {
  extern __shared__ float4 cs_sh[];                 // cosines and sines, see place_of
  __shared__ int64_t row_sh[kThreads];              // pool row; -1: padding, -2: no such row
  __shared__ int pos_sh[kThreads];
  __shared__ uint64_t turn_sh[kRopeMaxDim / 2];
  const int tid = threadIdx.x, sub = tid / lanes, nsub = kThreads / lanes, lane = tid % lanes;
  const int half = a.R / 2;
  const int kind = (int)blockIdx.x >= plan.start[2] ? 2 : (int)blockIdx.x >= plan.start[1] ? 1 : 0;
  const int tb = plan.tb[kind], splits = plan.splits[kind], block = blockIdx.x - plan.start[kind];
  const int64_t first = (int64_t)(block / splits) * tb;
  const int head0 = block % splits * plan.per[kind];
  const int heads = min(plan.per[kind], a.heads[kind] - head0);
  if (heads <= 0) return;                           // the last split may be empty
  const int here = a.n - first < tb ? (int)(a.n - first) : tb;   // tokens of this block
  const int units = a.dim / kUnit, turned = kPaired ? a.R / (2 * kUnit) : 0, start = a.at / kUnit;
  const bool norm = a.norm && kind != 2, rotate = half > 0 && kind != 2, quantised = kFp8 && kind != 0;
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
  // job: token `tok` of the block, head h of its heads
  const T* src0 = static_cast<const T*>(a.src[kind]) + first * a.src_stride[kind] + head0 * a.dim;
  const int64_t src_stride = a.src_stride[kind];
  Unit<T> next[kTasks][2];
  auto fetch = [&](int tok, int h) {
    if (tok >= here) return;
    const T* src = src0 + tok * src_stride + h * a.dim;
#pragma unroll
    for (int i = 0; i < kTasks; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (ua[i][e] >= 0) next[i][e].load(src + ua[i][e] * kUnit);
  };
  const int dtok = nsub / heads, dh = nsub - dtok * heads;
  int tok = sub / heads, h = sub - tok * heads;
  fetch(tok, h);
  const T* weight = norm ? static_cast<const T*>(a.weight[kind]) : nullptr;
  float w[kTasks][2][kUnit];
#pragma unroll
  for (int i = 0; i < kTasks; ++i)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int x = 0; x < kUnit; ++x) w[i][e][x] = 1.f;
      if (weight && ua[i][e] >= 0) {
        Unit<T> u;
        u.load(weight + ua[i][e] * kUnit);
        u.unpack(w[i][e]);
      }
    }

  // (lanes of a warp read different ones: not from the launch's constants each time)
  if (rotate)
    for (int i = tid; i < half; i += kThreads) turn_sh[i] = a.freq ? turn_of(a.freq[i]) : turns.t[i];
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
  // Cosine and sine of pair i of a token, in fours (cos, cos, sin, sin of two neighbouring
  // pairs) that the lanes of a head read side by side: 8 pairs of a lane's two units by
  // halves, 4 of either unit else.
  float* cs = reinterpret_cast<float*>(cs_sh);
  const int wide = a.halves ? turned : 2 * turned;   // lanes or units
  auto place_of = [&](int i) {
    if (!kPaired) return 2 * i;
    const int p = a.halves ? i / kUnit : i / (kUnit / 2), x = a.halves ? i % kUnit : i % (kUnit / 2);
    return ((x >> 1) * wide + p) * 4 + (x & 1);
  };
  if (rotate) {
    auto angle = [&](uint64_t turn, int k, float* to) {
      // the upper half of turn * pos modulo 2^64
      const uint32_t lo = (uint32_t)turn, pos = (uint32_t)pos_sh[k];
      const uint32_t phase = __umulhi(lo, pos) + (uint32_t)(turn >> 32) * pos - ((int)pos < 0 ? lo : 0u);
      float sn, cn;
      cos_sin(phase, cn, sn);
      to[0] = cn;
      to[kPaired ? 2 : 1] = sn;
    };
    int k = tid / half, i = tid - k * half;
    const int dk = kThreads / half, di = kThreads - dk * half;
    if (di == 0) {                               // a thread has the same pair of every token
      const uint64_t turn = turn_sh[i];
      float* to = cs + k * a.R + place_of(i);
#pragma unroll 2
      for (; k < here; k += dk, to += dk * a.R) angle(turn, k, to);
    } else {
      for (; k < here; k += dk, i += di) {
        if (i >= half) {
          i -= half;
          if (++k >= here) break;
        }
        angle(turn_sh[i], k, cs + k * a.R + place_of(i));
      }
    }
    __syncthreads();
  }

  const float inv_dim = 1.f / (float)a.dim;
  const int steps = (here * heads + nsub - 1) / nsub;   // the same for every thread (shuffles inside)
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
    tok += dtok;
    h += dh;
    if (h >= heads) h -= heads, ++tok;
    fetch(tok, h);
    const int64_t row = in ? row_sh[tok0] : -1;
    if (norm) {
      float sum[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < kTasks; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int x = 0; x < kUnit; x += 2) fma2(sum, f[i][e] + x, f[i][e] + x);
      float all = sum[0] + sum[1];
      for (int o = lanes / 2; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
      const float r = rsqrtf(fmaf(all, inv_dim, a.eps));
#pragma unroll
      for (int i = 0; i < kTasks; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int x = 0; x < kUnit; x += 2) {
            float rw[2] = {r, r};
            mul2(rw, w[i][e][x], w[i][e][x + 1]);
            mul2(f[i][e] + x, rw[0], rw[1]);
          }
    }
    if constexpr (!kPaired) {
      // pairs that do not fall on whole units: the partner's element through shared memory
      if (rotate) {
        float* y = cs + tb * a.R + sub * a.R;
        const float* c = cs + tok0 * a.R;
#pragma unroll
        for (int i = 0; i < kTasks; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int x = 0; x < kUnit; ++x) {
              const int d = ua[i][e] * kUnit + x - a.at;
              if (ua[i][e] >= 0 && d >= 0 && d < a.R) y[d] = f[i][e][x];
            }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kTasks; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int x = 0; x < kUnit; ++x) {
              const int d = ua[i][e] * kUnit + x - a.at;       // within the rotated dims
              if (!in || ua[i][e] < 0 || d < 0 || d >= a.R) continue;
              const bool second = a.halves ? d >= half : d & 1;
              const int k = a.halves ? (second ? d - half : d) : d >> 1;
              const float o = y[a.halves ? (second ? d - half : d + half) : d ^ 1] * c[2 * k + 1];
              f[i][e][x] = fmaf(f[i][e][x], c[2 * k], second ? o : -o);
            }
      }
    }
    if constexpr (kPaired) {
      if (rotate && in) {
        const float4* c4 = cs_sh + tok0 * (a.R / 4);
#pragma unroll
        for (int i = 0; i < kTasks; ++i) {
          const int p = lane + i * lanes;
          if (p >= turned) continue;
          if (a.halves) {
#pragma unroll
            for (int x = 0; x < kUnit; x += 2) {
              const float4 c = c4[(x >> 1) * wide + p];
              float* u = f[i][0] + x;
              float* v = f[i][1] + x;
              const float cn[2] = {c.x, c.y}, sn[2] = {c.z, c.w}, u0 = u[0], u1 = u[1];
              u[0] = fmaf(u[0], c.x, -(v[0] * c.z));
              u[1] = fmaf(u[1], c.y, -(v[1] * c.w));
              const float was[2] = {u0, u1};
              mul2(v, cn[0], cn[1]);
              fma2(v, was, sn);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int x = 0; x < kUnit; x += 4) {
                const float4 c = c4[(x >> 2) * wide + p + e * turned];
                float* u = f[i][e] + x;
                const float a0 = u[0], a1 = u[2];
                u[0] = fmaf(u[0], c.x, -(u[1] * c.z));
                u[1] = fmaf(u[1], c.x, a0 * c.z);
                u[2] = fmaf(u[2], c.y, -(u[3] * c.w));
                u[3] = fmaf(u[3], c.y, a1 * c.w);
              }
          }
        }
      }
    }
    __syncwarp();   // a head's lanes have read what an output in place overwrites
    float scale = 1.f;
    if (quantised) {
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
    if (quantised && lane == 0) a.scale[kind - 1][to * a.scale_stride + head0 + h0] = scale;
    const int64_t at = to * a.dst_stride[kind] + (head0 + h0) * a.dim;
#pragma unroll
    for (int i = 0; i < kTasks; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (ua[i][e] < 0) continue;
        if (quantised) {
          // the quotients as divide() forms them, two at a time
          const float inv = rcp_approx(scale), d = scale < INFINITY ? scale : 0.f, inv2[2] = {inv, inv};
#pragma unroll
          for (int x = 0; x < kUnit; x += 2) {
            float q[2] = {f[i][e][x], f[i][e][x + 1]};
            mul2(q, inv, inv);
            const float rest[2] = {fmaf(-q[0], d, f[i][e][x]), fmaf(-q[1], d, f[i][e][x + 1])};
            fma2(q, rest, inv2);
            f[i][e][x] = q[0], f[i][e][x + 1] = q[1];
          }
          uint32_t c[kUnit / 2];
#pragma unroll
          for (int x = 0; x < kUnit / 2; ++x)
            c[x] = __nv_cvt_float2_to_fp8x2(make_float2(f[i][e][2 * x], f[i][e][2 * x + 1]), __NV_SATFINITE, __NV_E4M3);
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.dst[kind]) + at + ua[i][e] * kUnit) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
        } else {
          Unit<T>::store(static_cast<T*>(a.dst[kind]) + at + ua[i][e] * kUnit, f[i][e]);
        }
      }
  }
}

template <typename T, int kTasks, bool kPaired>
int launch_shape(const HeadArgs& a, const Turns& turns, const Plan& plan, int lanes, bool fp8, cudaStream_t st, bool pdl) {
  const int tb = plan.tb[0] > plan.tb[1] ? plan.tb[0] : plan.tb[1];
  const size_t smem = (size_t)(tb + (kPaired ? 0 : kThreads / lanes)) * a.R * sizeof(float);
  return launch_kernel(fp8 ? heads_kernel<T, kTasks, kPaired, true> : heads_kernel<T, kTasks, kPaired, false>,
                       dim3((unsigned)plan.start[3]), dim3(kThreads), smem, st, pdl, a, turns, plan, lanes);
}

}  // namespace

int launch_heads(const HeadArgs& a, int dtype, bool fp8, double base, int num_sms, cudaStream_t st, bool pdl) {
  Turns turns;
  if (!a.freq && a.R > 0) {
    // every 16th by itself, so that no more than 16 roundings add up
    const double step = pow(base, -2.0 / a.R);
    double theta = 0.;
    for (int i = 0; i < a.R / 2; ++i, theta *= step) {
      if (i % 16 == 0) theta = 0.15915494309189535 * pow(base, -2.0 * i / a.R);   // 1 / (2 pi) of a turn per radian
      turns.t[i] = (uint64_t)(theta * 18446744073709551616.0);
    }
  }
  // whole units pair up where the rotated dims start on one and are a multiple of two
  const bool paired = a.at % kUnit == 0 && a.R % (2 * kUnit) == 0;
  const int units = a.dim / kUnit;
  const int tasks = paired ? a.R / (2 * kUnit) + (units - a.R / kUnit + 1) / 2 : (units + 1) / 2;
  int lanes = 1;
  while (lanes < tasks && lanes < 32) lanes *= 2;
  const int per = (tasks + lanes - 1) / lanes;   // 1, or 2 for heads of more than 64 units
  const int nsub = kThreads / lanes, kinds = (a.heads[0] > 0) + (a.heads[1] > 0) + (a.heads[2] > 0);
  const int64_t want = 8 * (int64_t)num_sms;     // blocks at least, if there is work for them
  Plan plan;
  int64_t start = 0;
  for (int k = 0; k < 3; ++k) {
    plan.start[k] = (int)start;
    plan.tb[k] = 0;
    if (a.heads[k] == 0) continue;
    const int H = a.heads[k], jobs = (H + nsub - 1) / nsub;   // turns of the block per token, at most
    // some jobs per lane, fewer tokens where there are not enough of them for the SMs, and then
    // the heads of a token in several blocks
    int64_t tb = (kJobs * nsub + H - 1) / H;
    const int64_t spread = (a.n * kinds + want - 1) / want;
    if (tb > spread) tb = spread;
    const int room = a.R > 0 && k != 2 ? 16384 / (a.R * (int)sizeof(float)) : kThreads;
    if (tb > room) tb = room;
    if (tb > kThreads) tb = kThreads;
    int64_t splits = tb > 1 ? 1 : want / (a.n * kinds);
    if (splits > jobs) splits = jobs;            // a job per lane at least
    if (splits < 1) splits = 1;
    plan.tb[k] = (int)tb;
    plan.splits[k] = (int)splits;
    plan.per[k] = (H + (int)splits - 1) / (int)splits;
    start += (a.n + tb - 1) / tb * splits;
    if (start > 0x7fffffff) return launch_fail("too many blocks", cudaErrorInvalidConfiguration);
  }
  plan.start[3] = (int)start;
  if (a.heads[2] == 0) plan.start[2] = plan.start[3];
  if (a.heads[1] == 0) plan.start[1] = plan.start[2];
#define CSA_HEADS(T)                                                                                          \
  (per == 1 ? paired ? launch_shape<T, 1, true>(a, turns, plan, lanes, fp8, st, pdl)                       \
                     : launch_shape<T, 1, false>(a, turns, plan, lanes, fp8, st, pdl)                      \
            : paired ? launch_shape<T, 2, true>(a, turns, plan, lanes, fp8, st, pdl)                       \
                     : launch_shape<T, 2, false>(a, turns, plan, lanes, fp8, st, pdl))
  return dtype == CSA_DTYPE_BF16 ? CSA_HEADS(__nv_bfloat16) : CSA_HEADS(float);
#undef CSA_HEADS
}

}  // namespace csa
