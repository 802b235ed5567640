// rotary.cu -- rotation of queries and keys by their positions.
//
// Of each head's first `rot` values, pairs (a, b) -- places (i, i + rot / 2), or
// neighbours (2 i, 2 i + 1) -- become gain (a cos t - b sin t, b cos t + a sin t),
// t the position times the frequency of pair i; the rest of the head stays.
//
// Bound by HBM: 2 bytes in and 2 out an element.  A thread owns up to eight pairs
// (four where they are neighbours) of a token for all heads of its slice, so that it
// finds their cosines and sines once (24,032 x 56 x 128: 106 us, 96% of the copy rate;
// a quarter of 28 heads of 256: 107 us; three tokens: 1.7 us, a launch).  A frequency is a number of turns a position
// in units of 2^-64, kept modulo one turn: the product with a position is exact
// modulo one turn in 64-bit integers, so that an angle is as exact at position
// 2^31 as at 1 (within 2^-33 turns of the frequency given, half a unit a position),
// for two integer multiplications; its upper half becomes fp32 and goes to
// sincospif.  Rotation is fp32, rounded to bf16 once.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/clef.h"
#include "clef_kernels.h"
#include "clef_ptx.cuh"
#include "kv_host.h"

namespace clef {

namespace {

constexpr float kFiniteGain = 3.4028234663852886e38f;

struct RotaryArgs {
    const uint16_t *x;
    uint16_t *out;
    const int32_t *pos;
    const int64_t *turns;
    int64_t ldx, ldx_head, ldo, ldo_head, tokens;
    int heads, slice;      // heads of the call, and of a row of CTAs
    int rot, tail;         // rotated values of a head, and those that only move (none in place)
    float gain;
};

__device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&p);
}

__device__ __forceinline__ void angle(const RotaryArgs &a, int32_t pos, int pair, float &c, float &s) {
    const uint64_t t = (uint64_t)(int64_t)pos * (uint64_t)a.turns[pair];
    // the upper half, signed: half turns in units of 2^-31
    sincospif((float)(int32_t)(uint32_t)(t >> 32) * 0x1p-31f, &s, &c);
    c *= a.gain;
    s *= a.gain;
}

// The pair of words (p, q) of two values each: p the first ones, q the second ones of their pairs.
__device__ __forceinline__ void turn(uint32_t &p, uint32_t &q, const float *c, const float *s) {
    const float a0 = lo(p), a1 = hi(p), b0 = lo(q), b1 = hi(q);
    p = pack2(fmaf(a0, c[0], -(b0 * s[0])), fmaf(a1, c[1], -(b1 * s[1])));
    q = pack2(fmaf(b0, c[0], a0 * s[0]), fmaf(b1, c[1], a1 * s[1]));
}

// A neighbouring pair in one word.
__device__ __forceinline__ uint32_t turn(uint32_t w, float c, float s) {
    const float a = lo(w), b = hi(w);
    return pack2(fmaf(a, c, -(b * s)), fmaf(b, c, a * s));
}

// V values (8, 4, 2 or 1), as words.
template <int V>
struct Piece {
    uint32_t w[V == 1 ? 1 : V / 2];

    __device__ __forceinline__ void load(const uint16_t *p) {
        if constexpr (V == 8) {
            const uint4 v = *reinterpret_cast<const uint4 *>(p);
            w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
        } else if constexpr (V == 4) {
            const uint2 v = *reinterpret_cast<const uint2 *>(p);
            w[0] = v.x; w[1] = v.y;
        } else if constexpr (V == 2) {
            w[0] = *reinterpret_cast<const uint32_t *>(p);
        } else {
            w[0] = *p;
        }
    }
    __device__ __forceinline__ void store(uint16_t *p) const {
        if constexpr (V == 8) *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else if constexpr (V == 4) *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        else if constexpr (V == 2) *reinterpret_cast<uint32_t *>(p) = w[0];
        else *p = (uint16_t)w[0];
    }
};

// Neighbouring pairs: a thread owns a piece of V values.  Otherwise two pieces: the first and the second values of V
// pairs, or two of those that only move.  Threads that rotate and threads that move share their loop, as a
// warp holds both.  Heads are taken kAhead at a time: their loads are on their way together.
template <int V, bool kNeighbours>
__global__ void __launch_bounds__(256) rotary_kernel(const RotaryArgs a) {
    constexpr int kPieces = kNeighbours ? 1 : 2, kPairs = kNeighbours ? V / 2 : V, kAhead = 4;
    const int units = a.rot / (kPieces * V), moved = (a.tail / V + kPieces - 1) / kPieces, per = units + moved;
    const int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x;
    const int64_t token = i / per;
    pdl_wait();
    if (token < a.tokens) {
        const int u = (int)(i - token * per), t = u - units;
        const bool turns = t < 0;
        // where its pieces start (a second one that there is not: the first once more)
        const int p0 = turns ? V * u : a.rot + V * t;
        const int p1 = turns ? p0 + a.rot / 2 : V * (t + moved) < a.tail ? p0 + V * moved : p0;
        const int h0 = blockIdx.y * a.slice, h1 = min(a.heads, h0 + a.slice);
        float c[kPairs], s[kPairs];
        if (turns) {
            const int32_t pos = a.pos[token];
#pragma unroll
            for (int k = 0; k < kPairs; ++k) angle(a, pos, kPairs * u + k, c[k], s[k]);
        }
        const uint16_t *x = a.x + token * a.ldx + h0 * a.ldx_head;
        uint16_t *out = a.out + token * a.ldo + h0 * a.ldo_head;
        for (int h = h0; h < h1; h += kAhead, x += kAhead * a.ldx_head, out += kAhead * a.ldo_head) {
            Piece<V> p[kAhead][kPieces];
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (h + k < h1) {
                    p[k][0].load(x + k * a.ldx_head + p0);
                    if (!kNeighbours) p[k][kPieces - 1].load(x + k * a.ldx_head + p1);
                }
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (h + k < h1) {
                    if (turns) {
                        if constexpr (kNeighbours) {
#pragma unroll
                            for (int j = 0; j < kPairs; ++j) p[k][0].w[j] = turn(p[k][0].w[j], c[j], s[j]);
                        } else if constexpr (V == 1) {
                            const uint32_t w = turn(p[k][0].w[0] | p[k][1].w[0] << 16, c[0], s[0]);
                            p[k][0].w[0] = w & 0xFFFFu;
                            p[k][1].w[0] = w >> 16;
                        } else {
#pragma unroll
                            for (int j = 0; j < V / 2; ++j) turn(p[k][0].w[j], p[k][1].w[j], c + 2 * j, s + 2 * j);
                        }
                    }
                    p[k][0].store(out + k * a.ldo_head + p0);
                    if (!kNeighbours) p[k][kPieces - 1].store(out + k * a.ldo_head + p1);
                }
        }
    }
    pdl_launch_dependents();
}

template <int V, bool kNeighbours>
int launch_rotary(RotaryArgs a, int sms, cudaStream_t st) {
    constexpr int kPieces = kNeighbours ? 1 : 2;
    const int per = a.rot / (kPieces * V) + (a.tail / V + kPieces - 1) / kPieces;
    const int64_t blocks = (a.tokens * per + 255) / 256;      // under 2^30 * 1024 / 256
    if (blocks > 0x7FFFFFFF) return kv_fail("too many tokens");
    // heads of a row of CTAs: all of them where the tokens alone give every SM its 2,048 threads, fewer otherwise
    const int64_t want = (int64_t)sms * 8;
    int rows = (int)(blocks >= want ? 1 : (want + blocks - 1) / blocks);
    if (rows > a.heads) rows = a.heads;
    a.slice = (a.heads + rows - 1) / rows;
    rows = (a.heads + a.slice - 1) / a.slice;
    const cudaError_t e = launch_kernel(rotary_kernel<V, kNeighbours>, dim3((unsigned)blocks, (unsigned)rows), dim3(256), 0, st, 1, true, a);
    return e == cudaSuccess ? CLEF_OK : internal_cuda_error(e, "rotary launch");
}

}  // namespace

}  // namespace clef

using namespace clef;

extern "C" int clef_rotary(const void *x, int64_t ldx, int64_t ldx_head, int64_t tokens, int heads, int dim, int rot,
                           int interleaved, const int32_t *pos, const int64_t *turns, float gain, void *out, int64_t ldo,
                           int64_t ldo_head, void *stream) {
    if (tokens < 0 || tokens > ((int64_t)1 << 30)) return kv_fail("tokens out of range");
    if (heads < 1 || heads > 1024) return kv_fail("heads must be in 1..1024");
    if (dim < 8 || dim > 1024 || dim % 8 != 0) return kv_fail("dim must be in 8..1024 and a multiple of 8");
    if (rot < 2 || rot > dim || rot % 2 != 0) return kv_fail("rot must be even and in 2..dim");
    if (!(gain >= -kFiniteGain && gain <= kFiniteGain)) return kv_fail("gain must be finite");
    for (const int64_t ld : {ldx, ldx_head, ldo, ldo_head})
        if (ld % 8 != 0 || ld < dim || ld > ((int64_t)1 << 40)) return kv_fail("pitches must be >= dim and multiples of 8");
    if (tokens == 0) return CLEF_OK;
    if (!x || !out || !pos || !turns) return kv_fail("null pointer");
    if (kv_misaligned(x, 16) || kv_misaligned(out, 16)) return kv_fail("x and out must be 16-byte aligned");
    if (kv_misaligned(pos, 4) || kv_misaligned(turns, 8)) return kv_fail("positions must be 4-byte and turns 8-byte aligned");
    const bool in_place = x == out;
    if (in_place && (ldx != ldo || ldx_head != ldo_head)) return kv_fail("in place, the pitches of x and out must agree");
    int sms = 0;
    unsigned int *status = nullptr;
    const int rc = internal_device(&sms, &status);
    if (rc) return rc;
    RotaryArgs a;
    a.x = static_cast<const uint16_t *>(x);
    a.out = static_cast<uint16_t *>(out);
    a.pos = pos;
    a.turns = turns;
    a.ldx = ldx;
    a.ldx_head = ldx_head;
    a.ldo = ldo;
    a.ldo_head = ldo_head;
    a.tokens = tokens;
    a.heads = heads;
    a.slice = heads;
    a.rot = rot;
    a.tail = in_place ? 0 : dim - rot;
    a.gain = gain;
    sms = internal_launch_sms(sms);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    // the widest pieces that the rotated part is whole ones of
    if (interleaved) return rot % 8 == 0 ? launch_rotary<8, true>(a, sms, st) : rot % 4 == 0 ? launch_rotary<4, true>(a, sms, st)
                                                                              : launch_rotary<2, true>(a, sms, st);
    return rot % 16 == 0 ? launch_rotary<8, false>(a, sms, st) : rot % 8 == 0 ? launch_rotary<4, false>(a, sms, st)
         : rot % 4 == 0 ? launch_rotary<2, false>(a, sms, st) : launch_rotary<1, false>(a, sms, st);
}
