// na_host.cuh -- host-side checks and tables shared by the C ABI's entry points
// (na_api.cu, latent_api.cu, pages_api.cu).
#pragma once

#include <math.h>

#include "na_internal.cuh"

constexpr double kPi = 3.14159265358979323846;

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The attention calls encode tensor maps with a driver call before they
// launch, and a driver call needs the device's context current on the calling
// thread.  The runtime binds it lazily (on a launch or a copy), so a thread
// whose first CUDA call is one of these may not have it yet: the current
// device's primary context is bound once per thread and device.
inline int bind_context()
{
    thread_local int bound = -1;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return NA_ERR_CUDA;
    if (dev != bound) {
        if (cudaSetDevice(dev) != cudaSuccess)
            return NA_ERR_CUDA;
        bound = dev;
    }
    return NA_OK;
}

inline int sm_count()
{
    // per device; an unreadable count plans for 152 SMs (the launches then
    // report the device error themselves)
    static std::atomic<int> cached[kMaxDevices];
    const int dev = current_device_index();
    if (dev >= 0) {
        const int n = cached[dev].load(std::memory_order_relaxed);
        if (n > 0)
            return n;
    }
    int d = 0, n = 0;
    if (cudaGetDevice(&d) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, d) != cudaSuccess || n <= 0)
        return 152;
    if (dev >= 0)
        cached[dev].store(n, std::memory_order_relaxed);
    return n;
}

// RoPE inverse frequencies in double (cortiq fns rope_inv_freq / yarn_inv_freq,
// with the rotary dimension as the exponent's denominator).
inline void rope_frequencies(const na_rope_params *r, int rd, double *out)
{
    const int half = rd / 2;
    if (!r->yarn) {
        for (int i = 0; i < half; i++)
            out[i] = pow(r->base, -2.0 * i / rd);
        return;
    }
    auto dim_at = [&](double rotations) {
        return rd * log(r->orig_max_pos / (rotations * 2.0 * kPi)) / (2.0 * log(r->base));
    };
    const int low = (int)fmax(floor(dim_at(r->beta_fast)), 0.0);
    const int high = (int)fmin(fmax(ceil(dim_at(r->beta_slow)), 0.0), (double)(half > 0 ? half - 1 : 0));
    const double span = (double)(high > low + 1 ? high - low : 1);
    for (int i = 0; i < half; i++) {
        const double plain = pow(r->base, -2.0 * i / rd);
        double ramp = (i > low ? i - low : 0) / span;
        ramp = ramp < 0.0 ? 0.0 : (ramp > 1.0 ? 1.0 : ramp);
        // ramp 0: keep the plain frequency; ramp 1: divide it by the factor.
        out[i] = plain * (1.0 - ramp) + (plain / r->factor) * ramp;
    }
}

// Multiplier on cos and sin: given value, else 1, else YaRN's 0.1 ln(factor) + 1.
inline double rope_attention_factor(const na_rope_params *r)
{
    if (r->attn_factor > 0.0)
        return r->attn_factor;
    if (r->yarn && r->factor > 1.0)
        return 0.1 * log(r->factor) + 1.0;
    return 1.0;
}

// The frequencies in turns, and the multiplier.  A step calls this with the same
// few parameters layer after layer, and 64 powers and divisions take longer than
// the launch (5 us of a call): each thread keeps its last table, by the values
// that determine it.
struct RopeTable {
    RopeTurns turns;
    float scale;
};

inline const RopeTable &rope_table(const na_rope_params *r, int rd)
{
    struct Kept {
        bool valid = false;
        na_rope_params r{};
        int rd = 0;
        RopeTable table{};
    };
    static thread_local Kept kept;
    const na_rope_params &k = kept.r;
    const bool same = kept.valid && kept.rd == rd && k.base == r->base && k.yarn == r->yarn &&
                      k.factor == r->factor && k.orig_max_pos == r->orig_max_pos &&
                      k.beta_fast == r->beta_fast && k.beta_slow == r->beta_slow &&
                      k.attn_factor == r->attn_factor;
    if (!same) {
        double inv_freq[64];
        rope_frequencies(r, rd, inv_freq);
        kept.table.turns = rope_turns_of(inv_freq, rd / 2);
        kept.table.scale = (float)rope_attention_factor(r);
        kept.r = *r;
        kept.rd = rd;
        kept.valid = true;
    }
    return kept.table;
}

inline int check_rope(const na_rope_params *r)
{
    if (!r || !(r->base > 1.0))
        return NA_ERR_INVALID_ARG;
    if (r->yarn && (!(r->factor > 0.0) || r->orig_max_pos <= 0 || !(r->beta_fast > 0.0) ||
                    !(r->beta_slow > 0.0)))
        return NA_ERR_INVALID_ARG;
    return NA_OK;
}

// log2 of a page size that the library takes (16, 32, 64 or 128), else -1.
inline int page_size_log(int page_size)
{
    for (int log = 4; log <= 7; log++)
        if (page_size == 1 << log)
            return log;
    return -1;
}
