// mt_seq_abi.cu -- the exported C ABI of the sequence-model calls
// (include/mt_scan.h): argument checks, then the launches of mt_embed.cu,
// mt_conv.cu and mt_ssm.cu.
#include <initializer_list>

#include "mt_seq.h"

using namespace mt;

namespace {

int act_size(int64_t dtype) { return dtype == MT_F32 ? 4 : dtype == MT_BF16 || dtype == MT_F16 ? 2 : 0; }

bool aligned(std::initializer_list<const void *> ps, uintptr_t to) {
    for (const void *p : ps)
        if ((uintptr_t)p % to != 0)
            return false;
    return true;
}
bool any_null(std::initializer_list<const void *> ps) {
    for (const void *p : ps)
        if (p == nullptr)
            return true;
    return false;
}
// Optional pointers that are absent are in reach.
bool in_device(std::initializer_list<const void *> ps, int dev) {
    for (const void *p : ps) {
        bool host = false;
        if (p != nullptr && (!ptr_reachable(p, dev, &host) || host))
            return false;
    }
    return true;
}
bool among(const void *p, std::initializer_list<const void *> ps) {
    for (const void *q : ps)
        if (p != nullptr && p == q)
            return true;
    return false;
}
// a * b * c * ... of sizes that are not negative, or -1 where it leaves int64's range by far
int64_t product(std::initializer_list<int64_t> xs) {
    int64_t r = 1;
    for (int64_t x : xs)
        if (x == 0)
            return 0;
    for (int64_t x : xs) {
        if (x < 0 || r > (INT64_MAX >> 8) / x)
            return -1;
        r *= x;
    }
    return r;
}
int done(cudaError_t e) { return e == cudaSuccess ? MT_OK : MT_ERR_CUDA; }

int conv_check(const mt_conv_args &a, bool tokens) {
    const int64_t len = tokens ? a.len : 1;
    if (a.batch < 0 || len < 0 || a.dim < 0 || a.width < 1 || a.width > 4 || a.nslots < 0)
        return MT_ERR_ARG;
    const int s = act_size(a.dtype);
    if (s == 0 || (a.wdtype != MT_F32 && a.wdtype != a.dtype))
        return MT_ERR_DTYPE;
    if (product({a.batch, len, a.dim, 8}) < 0 || product({a.nslots, a.width, a.dim, 8}) < 0)
        return MT_ERR_ARG;
    if (a.batch == 0 || a.dim == 0)
        return MT_OK;
    if (a.weight == nullptr || (len > 0 && a.x == nullptr))
        return MT_ERR_ARG;
    if (a.slots == nullptr && a.state != nullptr && a.nslots < a.batch)
        return MT_ERR_ARG;
    if (a.slots != nullptr && a.state == nullptr && a.width > 1)
        return MT_ERR_ARG;
    if (a.carry_in && a.state == nullptr && a.width > 1)
        return MT_ERR_ARG;
    const int w = a.wdtype == MT_F32 ? 4 : s;
    if (!aligned({a.x, a.state, a.out, a.dout, a.dx, a.dstate}, s) || !aligned({a.weight, a.bias}, w) ||
        !aligned({a.slots, a.lens, a.dweight, a.dbias}, 4) || !aligned({a.scratch}, 16))
        return MT_ERR_ALIGN;
    return MT_OK;
}

int ssm_check(const mt_ssm_args &a, bool tokens) {
    const int64_t len = tokens ? a.len : 1;
    if (a.batch < 0 || len < 0 || a.dim < 0 || a.nstate < 1 || a.nstate > 128 || a.groups < 1 || a.nslots < 0 ||
        a.dim % a.groups != 0)
        return MT_ERR_ARG;
    const int s = act_size(a.dtype);
    if (s == 0)
        return MT_ERR_DTYPE;
    if (product({a.batch, len, a.dim, 8}) < 0 || product({a.batch, len, a.groups, a.nstate, 8}) < 0 ||
        product({a.nslots, a.dim, a.nstate, 8}) < 0)
        return MT_ERR_ARG;
    if (a.batch == 0 || a.dim == 0)
        return MT_OK;
    if (a.A == nullptr || (len > 0 && any_null({a.u, a.delta, a.B, a.C})))
        return MT_ERR_ARG;
    if (a.slots == nullptr && a.state != nullptr && a.nslots < a.batch)
        return MT_ERR_ARG;
    if ((a.slots != nullptr || a.carry_in) && a.state == nullptr)
        return MT_ERR_ARG;
    if (!aligned({a.u, a.delta, a.z, a.B, a.C, a.out, a.dout, a.du, a.ddelta, a.dz, a.dB, a.dC}, s) ||
        !aligned({a.A, a.D, a.delta_bias, a.state, a.slots, a.lens, a.checkpoints, a.dA, a.dD, a.ddelta_bias, a.dfinal, a.dinit}, 4) ||
        !aligned({a.scratch}, 16))
        return MT_ERR_ALIGN;
    return MT_OK;
}

}  // namespace

extern "C" int mt_embed(const void *tokens, int64_t ntokens, int token_dtype, const void *table, int64_t vocab,
                        int64_t dim, int dtype, float scale, void *out, void *stream) {
    if (ntokens < 0 || vocab < 0 || dim < 0 || product({ntokens, dim, 8}) < 0 || product({vocab, dim, 8}) < 0)
        return MT_ERR_ARG;
    const int s = act_size(dtype);
    if (s == 0 || (token_dtype != MT_I32 && token_dtype != MT_I64))
        return MT_ERR_DTYPE;
    if (ntokens == 0 || dim == 0)
        return MT_OK;
    if (tokens == nullptr || out == nullptr || (table == nullptr && vocab > 0))
        return MT_ERR_ARG;
    if (among(out, {tokens, table}))
        return MT_ERR_ALIAS;
    if (!aligned({tokens}, token_dtype == MT_I64 ? 8 : 4) || !aligned({table, out}, s))
        return MT_ERR_ALIGN;
    Launch L;
    int dev = 0;
    if (!make_launch(stream, &L, &dev))
        return MT_ERR_CUDA;
    if (!in_device({tokens, table, out}, dev))
        return MT_ERR_MEMORY;
    return done(embed_launch(tokens, token_dtype == MT_I64, ntokens, table, vocab, dim, dtype, scale, out, L));
}

extern "C" int64_t mt_embed_grad_scratch_slots(int64_t ntokens, int64_t vocab, int64_t dim) {
    if (ntokens < 0 || vocab < 0 || dim < 0 || ntokens > INT32_MAX - 64 || vocab > INT32_MAX - 64 ||
        product({ntokens, dim, 8}) < 0 || product({vocab, dim, 8}) < 0 || dim > 65535 * 32)
        return -1;
    const EmbedGradPlan p = embed_grad_plan(ntokens, vocab, dim);
    return p.start_slots + 2 * p.order_slots + p.last_slots + p.partial_slots;
}

extern "C" int mt_embed_grad(const void *tokens, int64_t ntokens, int token_dtype, const void *dout, int dtype,
                             int64_t vocab, int64_t dim, float scale, void *dtable, int grad_dtype, int accumulate,
                             void *scratch, void *stream) {
    if (mt_embed_grad_scratch_slots(ntokens, vocab, dim) < 0)
        return MT_ERR_ARG;
    const int s = act_size(dtype), sg = act_size(grad_dtype);
    if (s == 0 || (token_dtype != MT_I32 && token_dtype != MT_I64) || (grad_dtype != MT_F32 && grad_dtype != dtype))
        return MT_ERR_DTYPE;
    if (vocab == 0 || dim == 0 || (accumulate && ntokens == 0))
        return MT_OK;
    if (dtable == nullptr || scratch == nullptr || (ntokens > 0 && any_null({tokens, dout})))
        return MT_ERR_ARG;
    if (among(dtable, {tokens, dout, scratch}) || among(scratch, {tokens, dout}))
        return MT_ERR_ALIAS;
    if (!aligned({tokens}, token_dtype == MT_I64 ? 8 : 4) || !aligned({dout}, s) || !aligned({dtable}, sg) ||
        !aligned({scratch}, 16))
        return MT_ERR_ALIGN;
    Launch L;
    int dev = 0;
    if (!make_launch(stream, &L, &dev))
        return MT_ERR_CUDA;
    if (!in_device({tokens, dout, dtable, scratch}, dev))
        return MT_ERR_MEMORY;
    return done(embed_grad_launch(tokens, token_dtype == MT_I64, ntokens, dout, dtype, vocab, dim, scale, dtable, grad_dtype,
                                  accumulate != 0, static_cast<uint64_t *>(scratch), L));
}

extern "C" int mt_causal_conv(const mt_conv_args *args, void *stream) {
    if (args == nullptr)
        return MT_ERR_ARG;
    const mt_conv_args &a = *args;
    const int bad = conv_check(a, true);
    if (bad != MT_OK || a.batch == 0 || a.dim == 0)
        return bad;
    if (a.len > 0 && a.out == nullptr)
        return MT_ERR_ARG;
    if (among(a.out, {a.x, a.weight, a.bias, a.state}) || among(a.state, {a.x, a.weight, a.bias}))
        return MT_ERR_ALIAS;
    Launch L;
    int dev = 0;
    if (!make_launch(stream, &L, &dev))
        return MT_ERR_CUDA;
    if (!in_device({a.x, a.weight, a.bias, a.state, a.slots, a.lens, a.out}, dev))
        return MT_ERR_MEMORY;
    return done(conv_launch(a, L));
}

extern "C" int mt_causal_conv_step(const mt_conv_args *args, void *stream) {
    if (args == nullptr)
        return MT_ERR_ARG;
    const mt_conv_args &a = *args;
    const int bad = conv_check(a, false);
    if (bad != MT_OK || a.batch == 0 || a.dim == 0)
        return bad;
    if (a.out == nullptr || (a.state == nullptr && a.width > 1))
        return MT_ERR_ARG;
    if (among(a.out, {a.x, a.weight, a.bias, a.state}) || among(a.state, {a.x, a.weight, a.bias}))
        return MT_ERR_ALIAS;
    Launch L;
    int dev = 0;
    if (!make_launch(stream, &L, &dev))
        return MT_ERR_CUDA;
    if (!in_device({a.x, a.weight, a.bias, a.state, a.slots, a.out}, dev))
        return MT_ERR_MEMORY;
    return done(conv_step_launch(a, L));
}

extern "C" int64_t mt_causal_conv_grad_scratch_slots(int64_t batch, int64_t len, int64_t dim, int64_t width) {
    if (batch < 0 || len < 0 || dim < 0 || width < 1 || width > 4 || product({batch, len, dim, 16}) < 0 ||
        product({batch, dim, 16}) < 0)
        return -1;
    return conv_grad_scratch_slots(batch, len, dim, width);
}

extern "C" int mt_causal_conv_grad(const mt_conv_args *args, void *stream) {
    if (args == nullptr)
        return MT_ERR_ARG;
    const mt_conv_args &a = *args;
    const int bad = conv_check(a, true);
    if (bad != MT_OK || a.dim == 0)
        return bad;
    if (a.slots != nullptr || a.dweight == nullptr)
        return MT_ERR_ARG;
    if (a.batch > 0 && (a.scratch == nullptr || (a.len > 0 && any_null({a.dout, a.dx}))))
        return MT_ERR_ARG;
    for (const void *p : {(const void *)a.dx, (const void *)a.dweight, (const void *)a.dbias, (const void *)a.dstate, (const void *)a.scratch})
        if (among(p, {a.x, a.weight, a.bias, a.state, a.dout}))
            return MT_ERR_ALIAS;
    Launch L;
    int dev = 0;
    if (!make_launch(stream, &L, &dev))
        return MT_ERR_CUDA;
    if (!in_device({a.x, a.weight, a.bias, a.state, a.lens, a.dout, a.dx, a.dweight, a.dbias, a.dstate, a.scratch}, dev))
        return MT_ERR_MEMORY;
    return done(conv_grad_launch(a, L));
}

extern "C" int64_t mt_selective_scan_scratch_slots(int64_t batch, int64_t len, int64_t dim, int64_t nstate,
                                                   int64_t groups, int grad) {
    if (batch < 0 || len < 0 || dim < 0 || nstate < 1 || nstate > 128 || groups < 1 || dim % groups != 0 ||
        product({batch, len, dim, nstate, 16}) < 0 || product({batch, len, groups, nstate, 16}) < 0 ||
        product({batch, dim, nstate, 16}) < 0)
        return -1;
    int64_t most = 0;  // of the plans with live lengths and without
    for (const bool lens : {false, true}) {
        const SsmPlan p = ssm_plan(batch, len, dim, nstate, groups, grad != 0, lens);
        const int64_t slots = p.carry_slots + p.decay_slots + p.shared_slots + p.param_slots;
        most = slots > most ? slots : most;
    }
    return most;
}

extern "C" int64_t mt_selective_scan_checkpoint_slots(int64_t batch, int64_t len, int64_t dim, int64_t nstate) {
    if (batch < 0 || len < 0 || dim < 0 || nstate < 1 || nstate > 128 || product({batch, len, dim, nstate, 16}) < 0)
        return -1;
    return (batch * ((len + kSsmTile - 1) / kSsmTile) * dim * nstate + 1) / 2;
}

extern "C" int mt_selective_scan(const mt_ssm_args *args, void *stream) {
    if (args == nullptr)
        return MT_ERR_ARG;
    const mt_ssm_args &a = *args;
    const int bad = ssm_check(a, true);
    if (bad != MT_OK || a.batch == 0 || a.dim == 0)
        return bad;
    const int64_t slots = mt_selective_scan_scratch_slots(a.batch, a.len, a.dim, a.nstate, a.groups, 0);
    if ((a.len > 0 && a.out == nullptr) || slots < 0 || (slots > 0 && a.scratch == nullptr) ||
        (a.checkpoints != nullptr && a.slots != nullptr))
        return MT_ERR_ARG;
    for (const void *p : {(const void *)a.out, (const void *)a.state, (const void *)a.checkpoints, (const void *)a.scratch})
        if (among(p, {a.u, a.delta, a.z, a.B, a.C, a.A, a.D, a.delta_bias}))
            return MT_ERR_ALIAS;
    if (among(a.out, {a.state, a.checkpoints, a.scratch}) || among(a.state, {a.checkpoints, a.scratch}))
        return MT_ERR_ALIAS;
    Launch L;
    int dev = 0;
    if (!make_launch(stream, &L, &dev))
        return MT_ERR_CUDA;
    if (!in_device({a.u, a.delta, a.z, a.B, a.C, a.A, a.D, a.delta_bias, a.state, a.slots, a.lens, a.out, a.checkpoints, a.scratch}, dev))
        return MT_ERR_MEMORY;
    return done(ssm_launch(a, L));
}

extern "C" int mt_selective_scan_step(const mt_ssm_args *args, void *stream) {
    if (args == nullptr)
        return MT_ERR_ARG;
    const mt_ssm_args &a = *args;
    const int bad = ssm_check(a, false);
    if (bad != MT_OK || a.batch == 0 || a.dim == 0)
        return bad;
    if (any_null({a.out, a.state}))
        return MT_ERR_ARG;
    if (among(a.out, {a.u, a.delta, a.z, a.B, a.C, a.A, a.D, a.delta_bias, a.state}) ||
        among(a.state, {a.u, a.delta, a.z, a.B, a.C, a.A, a.D, a.delta_bias}))
        return MT_ERR_ALIAS;
    Launch L;
    int dev = 0;
    if (!make_launch(stream, &L, &dev))
        return MT_ERR_CUDA;
    if (!in_device({a.u, a.delta, a.z, a.B, a.C, a.A, a.D, a.delta_bias, a.state, a.slots, a.out}, dev))
        return MT_ERR_MEMORY;
    return done(ssm_step_launch(a, L));
}

extern "C" int mt_selective_scan_grad(const mt_ssm_args *args, void *stream) {
    if (args == nullptr)
        return MT_ERR_ARG;
    mt_ssm_args a = *args;
    a.state = nullptr;
    a.carry_in = 0;
    const int bad = ssm_check(a, true);
    if (bad != MT_OK || a.dim == 0)
        return bad;
    const bool work = a.batch > 0 && a.len > 0;
    if (a.dA == nullptr || mt_selective_scan_scratch_slots(a.batch, a.len, a.dim, a.nstate, a.groups, 1) < 0)
        return MT_ERR_ARG;
    if (a.batch > 0 && a.scratch == nullptr)
        return MT_ERR_ARG;
    if (work && (any_null({a.dout, a.checkpoints, a.du, a.ddelta, a.dB, a.dC}) || (a.z != nullptr && a.dz == nullptr)))
        return MT_ERR_ARG;
    for (const void *p : {(const void *)a.du, (const void *)a.ddelta, (const void *)a.dz, (const void *)a.dB, (const void *)a.dC, (const void *)a.dA,
                          (const void *)a.dD, (const void *)a.ddelta_bias, (const void *)a.dinit, (const void *)a.scratch})
        if (among(p, {a.u, a.delta, a.z, a.B, a.C, a.A, a.D, a.delta_bias, a.dout, a.checkpoints, a.dfinal}))
            return MT_ERR_ALIAS;
    Launch L;
    int dev = 0;
    if (!make_launch(stream, &L, &dev))
        return MT_ERR_CUDA;
    if (!in_device({a.u, a.delta, a.z, a.B, a.C, a.A, a.D, a.delta_bias, a.lens, a.checkpoints, a.scratch, a.dout}, dev) ||
        !in_device({a.du, a.ddelta, a.dz, a.dB, a.dC, a.dA, a.dD, a.ddelta_bias, a.dfinal, a.dinit}, dev))
        return MT_ERR_MEMORY;
    return done(ssm_grad_launch(a, L));
}
