// rotary.cu -- rotation of queries and keys by their positions.
//
// Of each head's first `rot` values, pairs (a, b) -- places (i, i + rot / 2), or
// neighbours (2 i, 2 i + 1) -- become gain (a cos t - b sin t, b cos t + a sin t),
// t the position times the frequency of pair i; the rest of the head stays.
//
// Bound by HBM: 2 bytes in and 2 out an element.  A thread owns eight pairs (four
// where they are neighbours) of a token for all heads of its slice, so that it
// finds their cosines and sines once.  A frequency is a number of turns a position
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
    int pairs;             // pairs of a head
    int units, tail;       // pieces of a token: of pairs, and of values that only move (none in place)
    int rot;
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

// Pieces of 16 bytes: two of a head's halves, or one of neighbouring pairs.
template <bool kNeighbours>
__global__ void __launch_bounds__(256) rotary_kernel(const RotaryArgs a) {
    const int per = a.units + a.tail;
    const int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x;
    const int64_t token = i / per;
    pdl_wait();
    if (token < a.tokens) {
        const int u = (int)(i - token * per);
        const int h0 = blockIdx.y * a.slice, h1 = min(a.heads, h0 + a.slice);
        const uint16_t *x = a.x + token * a.ldx;
        uint16_t *out = a.out + token * a.ldo;
        if (u >= a.units) {
            const int at = a.rot + 8 * (u - a.units);
#pragma unroll 4
            for (int h = h0; h < h1; ++h)
                *reinterpret_cast<uint4 *>(out + h * a.ldo_head + at) = *reinterpret_cast<const uint4 *>(x + h * a.ldx_head + at);
        } else if (kNeighbours) {
            const int32_t pos = a.pos[token];
            float c[4], s[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) angle(a, pos, 4 * u + k, c[k], s[k]);
#pragma unroll 4
            for (int h = h0; h < h1; ++h) {
                uint4 w = *reinterpret_cast<const uint4 *>(x + h * a.ldx_head + 8 * u);
                w = make_uint4(turn(w.x, c[0], s[0]), turn(w.y, c[1], s[1]), turn(w.z, c[2], s[2]), turn(w.w, c[3], s[3]));
                *reinterpret_cast<uint4 *>(out + h * a.ldo_head + 8 * u) = w;
            }
        } else {
            const int32_t pos = a.pos[token];
            float c[8], s[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) angle(a, pos, 8 * u + k, c[k], s[k]);
#pragma unroll 4
            for (int h = h0; h < h1; ++h) {
                const uint16_t *from = x + h * a.ldx_head + 8 * u;
                uint16_t *to = out + h * a.ldo_head + 8 * u;
                uint4 p = *reinterpret_cast<const uint4 *>(from), q = *reinterpret_cast<const uint4 *>(from + a.pairs);
                turn(p.x, q.x, c, s);
                turn(p.y, q.y, c + 2, s + 2);
                turn(p.z, q.z, c + 4, s + 4);
                turn(p.w, q.w, c + 6, s + 6);
                *reinterpret_cast<uint4 *>(to) = p;
                *reinterpret_cast<uint4 *>(to + a.pairs) = q;
            }
        }
    }
    pdl_launch_dependents();
}

// Pieces of one pair or one value, for heads whose rotated part does not end between pieces of 16 bytes.
__global__ void __launch_bounds__(256) rotary_single_kernel(const RotaryArgs a, int interleaved) {
    const int per = a.units + a.tail;
    const int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x;
    const int64_t token = i / per;
    pdl_wait();
    if (token < a.tokens) {
        const int u = (int)(i - token * per);
        const int h0 = blockIdx.y * a.slice, h1 = min(a.heads, h0 + a.slice);
        const uint16_t *x = a.x + token * a.ldx;
        uint16_t *out = a.out + token * a.ldo;
        if (u >= a.units) {
            const int at = a.rot + u - a.units;
            for (int h = h0; h < h1; ++h) out[h * a.ldo_head + at] = x[h * a.ldx_head + at];
        } else {
            float c, s;
            angle(a, a.pos[token], u, c, s);
            const int first = interleaved ? 2 * u : u, second = interleaved ? 2 * u + 1 : u + a.pairs;
#pragma unroll 4
            for (int h = h0; h < h1; ++h) {
                const uint32_t w = turn(x[h * a.ldx_head + first] | (uint32_t)x[h * a.ldx_head + second] << 16, c, s);
                out[h * a.ldo_head + first] = (uint16_t)w;
                out[h * a.ldo_head + second] = (uint16_t)(w >> 16);
            }
        }
    }
    pdl_launch_dependents();
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
    a.pairs = rot / 2;
    a.rot = rot;
    a.gain = gain;
    const int width = interleaved ? 8 : 16;       // values of a piece of pairs
    const bool whole = rot % width == 0;
    a.units = whole ? rot / width : rot / 2;
    a.tail = in_place ? 0 : whole ? (dim - rot) / 8 : dim - rot;
    const int64_t blocks = (tokens * (a.units + a.tail) + 255) / 256;   // under 2^30 * 1024 / 256
    if (blocks > 0x7FFFFFFF) return kv_fail("too many tokens");
    // heads of a row of CTAs: all of them where the tokens alone give every SM its 2,048 threads, fewer otherwise
    const int64_t want = (int64_t)internal_launch_sms(sms) * 8;
    int rows = (int)(blocks >= want ? 1 : (want + blocks - 1) / blocks);
    if (rows > heads) rows = heads;
    a.slice = (heads + rows - 1) / rows;
    rows = (heads + a.slice - 1) / a.slice;
    const dim3 grid((unsigned)blocks, (unsigned)rows);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (!whole) e = launch_kernel(rotary_single_kernel, grid, dim3(256), 0, st, 1, true, a, interleaved ? 1 : 0);
    else if (interleaved) e = launch_kernel(rotary_kernel<true>, grid, dim3(256), 0, st, 1, true, a);
    else e = launch_kernel(rotary_kernel<false>, grid, dim3(256), 0, st, 1, true, a);
    return e == cudaSuccess ? CLEF_OK : internal_cuda_error(e, "rotary launch");
}
