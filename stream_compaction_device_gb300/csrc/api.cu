// C ABI of the devscan library: argument validation, the per-stream
// workspace, and dispatch to the kernels.  Declared in include/devscan.h.
#include <algorithm>
#include <atomic>
#include <cstdint>
#include <map>
#include <memory>
#include <mutex>
#include <new>
#include <numeric>
#include <utility>
#include <vector>

#include "../../include/devscan.h"
#include "../../include/devscan_measure.h"
#include "core.cuh"
#include "launch.h"

namespace devscan {
namespace {

// Polls of a look-back wait before it gives up (each poll after the fourth
// sleeps 32-256 ns, so the bound is well above any legitimate wait: a
// predecessor tile only has to load and reduce its own data).
constexpr unsigned kSpinLimit = 1u << 21;

// Largest tile count a workspace may hold: its capacity doubles from 1,024
// in 64-bit arithmetic up to this power of two, so no size can wrap it.
constexpr size_t kMaxTiles = size_t(1) << 31;
constexpr size_t kMaxScanN = kMaxTiles * kScanTile;

// The inter-block carry strategy of the calling thread's calls (kCarry*),
// set only through devscan_measure_set_carry_mode (include/devscan_measure.h):
// one thread choosing a path for a measurement leaves every other thread's
// calls on the default.
thread_local int t_carry_mode = kCarryDefault;
int carry_mode() { return t_carry_mode; }

struct Slot {
    void *base = nullptr;
    size_t bytes = 0;
    Workspace ws;
    void *extra = nullptr;   // per-stream scratch, of what the largest call so far asked for
    size_t extra_bytes = 0;
    std::shared_ptr<std::mutex> calls = std::make_shared<std::mutex>();   // held by one call at a time
};

using SlotKey = std::pair<int, uintptr_t>;   // device, stream

std::mutex g_mutex;   // of the maps
std::map<SlotKey, Slot> g_slots;
std::map<int, int> g_num_sms;

// A call's hold on its stream's slot, from finding it to the call's last
// launch.  A call's launches hand each other what is in the workspace and the
// scratch, so another thread's call on the same stream must not come between
// them, nor free a scratch that it outgrows before they are queued.
struct Hold {
    std::shared_ptr<std::mutex> calls;   // outlives the slot, which another thread may release
    std::unique_lock<std::mutex> lock;
};

// Holds the slot of `key` and returns it; null if there is none and none is
// to be made.
Slot *hold_slot(const SlotKey &key, bool make, Hold *hold)
{
    for (;;) {
        hold->lock = {};
        {
            std::lock_guard<std::mutex> lock(g_mutex);
            const auto it = make ? g_slots.try_emplace(key).first : g_slots.find(key);
            if (it == g_slots.end()) return nullptr;
            hold->calls = it->second.calls;
        }
        hold->lock = std::unique_lock<std::mutex>(*hold->calls);
        std::lock_guard<std::mutex> lock(g_mutex);
        const auto it = g_slots.find(key);
        if (it != g_slots.end() && it->second.calls == hold->calls) return &it->second;   // else released meanwhile
    }
}

constexpr size_t kStateBytes = 256;

size_t layout_bytes(unsigned capacity)
{
    // state | status[capacity] | group status[capacity / 32] | never_published[2] | tile_sums[capacity]
    return kStateBytes + static_cast<size_t>(capacity) * 8 + static_cast<size_t>(capacity / 32) * 8 + 16 +
           static_cast<size_t>(capacity) * 4 + 256;
}

devscan_status from_cuda(cudaError_t e) { return e == cudaSuccess ? DEVSCAN_OK : DEVSCAN_ERR_CUDA; }

// Finds (or grows) the workspace of (current device, stream) so that it holds
// at least `tiles` tile slots.  Growth frees the old block and allocates a
// new one stream-ordered, then zeroes it on the stream, so calls already
// queued on the stream finish with the old block first.  The workspace is the
// call's while it has `hold`.
devscan_status acquire(cudaStream_t stream, unsigned tiles, Workspace *out, Hold *hold)
try {
    static_assert(sizeof(DevState) <= kStateBytes, "device state must fit its slot");
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return DEVSCAN_ERR_CUDA;
    if (tiles > kMaxTiles) return DEVSCAN_ERR_INVALID;
    const SlotKey key{dev, reinterpret_cast<uintptr_t>(stream)};
    Slot &slot = *hold_slot(key, true, hold);
    std::lock_guard<std::mutex> lock(g_mutex);
    auto sms = g_num_sms.find(dev);
    if (sms == g_num_sms.end()) {
        int count = 0;
        if (cudaDeviceGetAttribute(&count, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return DEVSCAN_ERR_CUDA;
        sms = g_num_sms.emplace(dev, count).first;
    }
    if (slot.base == nullptr || slot.ws.capacity < tiles) {
        size_t cap = 1024;
        while (cap < tiles) cap *= 2;   // at most kMaxTiles = 2^31
        const unsigned capacity = static_cast<unsigned>(cap);
        const size_t bytes = layout_bytes(capacity);
        if (slot.base != nullptr) {
            if (cudaFreeAsync(slot.base, stream) != cudaSuccess) return DEVSCAN_ERR_CUDA;
            slot.base = nullptr;
        }
        void *base = nullptr;
        const cudaError_t e = cudaMallocAsync(&base, bytes, stream);
        if (e != cudaSuccess) {
            (void)cudaGetLastError();
            g_slots.erase(key);
            return e == cudaErrorMemoryAllocation ? DEVSCAN_ERR_NOMEM : DEVSCAN_ERR_CUDA;
        }
        if (cudaMemsetAsync(base, 0, bytes, stream) != cudaSuccess) return DEVSCAN_ERR_CUDA;
        char *p = static_cast<char *>(base);
        slot.base = base;
        slot.bytes = bytes;
        slot.ws.state = reinterpret_cast<DevState *>(p);
        slot.ws.status = reinterpret_cast<unsigned long long *>(p + kStateBytes);
        slot.ws.never_published = slot.ws.status + capacity + capacity / 32;
        slot.ws.tile_sums = reinterpret_cast<uint32_t *>(slot.ws.never_published + 2);
        slot.ws.capacity = capacity;
    }
    slot.ws.num_sms = sms->second;
    *out = slot.ws;
    return DEVSCAN_OK;
} catch (const std::bad_alloc &) {
    return DEVSCAN_ERR_NOMEM;
}

// Per-stream scratch of at least `bytes`, grown stream-ordered like the
// workspace (by a call that holds the slot: call acquire() first).
devscan_status acquire_extra(cudaStream_t stream, size_t bytes, void **out)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return DEVSCAN_ERR_CUDA;
    std::lock_guard<std::mutex> lock(g_mutex);
    auto it = g_slots.find({dev, reinterpret_cast<uintptr_t>(stream)});
    if (it == g_slots.end()) return DEVSCAN_ERR_CUDA;
    Slot &slot = it->second;
    if (slot.extra_bytes < bytes) {
        if (slot.extra != nullptr && cudaFreeAsync(slot.extra, stream) != cudaSuccess) return DEVSCAN_ERR_CUDA;
        slot.extra = nullptr;
        slot.extra_bytes = 0;
        void *p = nullptr;
        const cudaError_t e = cudaMallocAsync(&p, bytes, stream);
        if (e != cudaSuccess) {
            (void)cudaGetLastError();
            return e == cudaErrorMemoryAllocation ? DEVSCAN_ERR_NOMEM : DEVSCAN_ERR_CUDA;
        }
        slot.extra = p;
        slot.extra_bytes = bytes;
    }
    *out = slot.extra;
    return DEVSCAN_OK;
}

bool overlaps(const void *a, size_t abytes, const void *b, size_t bbytes)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + bbytes && y < x + abytes;
}

devscan_status scan_common(ElemType type, bool inclusive, const void *in, void *out, size_t n, devscan_op op,
                           cudaStream_t stream, const void *carry_in = nullptr)
{
    if (op != DEVSCAN_OP_ADD && op != DEVSCAN_OP_MAX && op != DEVSCAN_OP_XOR) return DEVSCAN_ERR_INVALID;
    if (type == ElemType::F32 && op == DEVSCAN_OP_XOR) return DEVSCAN_ERR_UNSUPPORTED;
    if (n == 0) return DEVSCAN_OK;
    if (in == nullptr || out == nullptr) return DEVSCAN_ERR_INVALID;
    if (reinterpret_cast<uintptr_t>(in) % 4 != 0 || reinterpret_cast<uintptr_t>(out) % 4 != 0)
        return DEVSCAN_ERR_INVALID;
    if (n > kMaxScanN) return DEVSCAN_ERR_INVALID;
    if (carry_in != nullptr &&
        (reinterpret_cast<uintptr_t>(carry_in) % 4 != 0 || overlaps(carry_in, 4, out, n * 4)))
        return DEVSCAN_ERR_INVALID;
    const unsigned tiles = tiles_for(n, kScanTile);
    Workspace ws;
    Hold hold;
    const devscan_status st = acquire(stream, tiles, &ws, &hold);
    if (st != DEVSCAN_OK) return st;
    const bool aligned = reinterpret_cast<uintptr_t>(in) % 16 == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0;
    const int carry = carry_mode();
    return from_cuda(launch_scan(type, static_cast<int>(op), inclusive, in, out, n, aligned, carry, ws,
                                 kSpinLimit, stream, carry_in));
}

// Host arrays in, host array out: the input is copied into the caller's
// device buffer, scanned there into the second device buffer, and the result
// copied back, all ordered on `stream`.
devscan_status scan_host_common(ElemType type, bool inclusive, const void *h_in, void *h_out, size_t n,
                                devscan_op op, void *d_in, void *d_out, cudaStream_t stream)
{
    if (op != DEVSCAN_OP_ADD && op != DEVSCAN_OP_MAX && op != DEVSCAN_OP_XOR) return DEVSCAN_ERR_INVALID;
    if (type == ElemType::F32 && op == DEVSCAN_OP_XOR) return DEVSCAN_ERR_UNSUPPORTED;
    if (n == 0) return DEVSCAN_OK;
    if (h_in == nullptr || h_out == nullptr || d_in == nullptr || d_out == nullptr) return DEVSCAN_ERR_INVALID;
    if (n > kMaxScanN) return DEVSCAN_ERR_INVALID;
    const size_t bytes = n * 4;
    if (overlaps(d_in, bytes, d_out, bytes) && d_in != d_out) return DEVSCAN_ERR_INVALID;
    if (cudaMemcpyAsync(d_in, h_in, bytes, cudaMemcpyHostToDevice, stream) != cudaSuccess) return DEVSCAN_ERR_CUDA;
    const devscan_status st = scan_common(type, inclusive, d_in, d_out, n, op, stream);
    if (st != DEVSCAN_OK) return st;
    return from_cuda(cudaMemcpyAsync(h_out, d_out, bytes, cudaMemcpyDeviceToHost, stream));
}

devscan_status reduce_common(ElemType type, const void *in, size_t n, devscan_op op, void *total,
                             cudaStream_t stream)
{
    if (op != DEVSCAN_OP_ADD && op != DEVSCAN_OP_MAX && op != DEVSCAN_OP_XOR) return DEVSCAN_ERR_INVALID;
    if (type == ElemType::F32 && op == DEVSCAN_OP_XOR) return DEVSCAN_ERR_UNSUPPORTED;
    if (total == nullptr || reinterpret_cast<uintptr_t>(total) % 4 != 0) return DEVSCAN_ERR_INVALID;
    if (n > kMaxScanN) return DEVSCAN_ERR_INVALID;
    if (n > 0 && (in == nullptr || reinterpret_cast<uintptr_t>(in) % 4 != 0 || overlaps(total, 4, in, n * 4)))
        return DEVSCAN_ERR_INVALID;
    Workspace ws;
    Hold hold;
    const devscan_status st = acquire(stream, 1, &ws, &hold);
    if (st != DEVSCAN_OK) return st;
    return from_cuda(launch_reduce(type, static_cast<int>(op), in, n, total, ws, stream));
}

devscan_status segscan_common(ElemType type, bool inclusive, const void *in, const uint8_t *heads, void *out,
                              size_t n, devscan_op op, cudaStream_t stream)
{
    if (op != DEVSCAN_OP_ADD && op != DEVSCAN_OP_MAX && op != DEVSCAN_OP_XOR) return DEVSCAN_ERR_INVALID;
    if (type == ElemType::F32 && op == DEVSCAN_OP_XOR) return DEVSCAN_ERR_UNSUPPORTED;
    if (n == 0) return DEVSCAN_OK;
    if (in == nullptr || heads == nullptr || out == nullptr) return DEVSCAN_ERR_INVALID;
    if (reinterpret_cast<uintptr_t>(in) % 4 != 0 || reinterpret_cast<uintptr_t>(out) % 4 != 0)
        return DEVSCAN_ERR_INVALID;
    if (n > kMaxScanN) return DEVSCAN_ERR_INVALID;
    if (overlaps(heads, n, out, n * 4) || (in != out && overlaps(in, n * 4, out, n * 4))) return DEVSCAN_ERR_INVALID;
    Workspace ws;
    Hold hold;
    const devscan_status st = acquire(stream, tiles_for(n, kScanTile), &ws, &hold);
    if (st != DEVSCAN_OK) return st;
    return from_cuda(launch_segscan(type, static_cast<int>(op), inclusive, in, heads, out, n,
                                    carry_mode(), ws, kSpinLimit, stream));
}

bool misaligned(const void *p, size_t size) { return reinterpret_cast<uintptr_t>(p) % size != 0; }

// A buffer of a call; null for an optional argument, or of no bytes.
struct Span {
    const void *p;
    size_t bytes;
    bool empty() const { return p == nullptr || bytes == 0; }
};

// Whether one of the buffers that a call writes overlaps another of its
// buffers.
template <size_t W, size_t R>
bool written_overlap(const Span (&written)[W], const Span (&read)[R])
{
    for (size_t i = 0; i < W; ++i) {
        if (written[i].empty()) continue;
        for (size_t j = i + 1; j < W; ++j)
            if (!written[j].empty() && overlaps(written[i].p, written[i].bytes, written[j].p, written[j].bytes))
                return true;
        for (size_t j = 0; j < R; ++j)
            if (!read[j].empty() && overlaps(written[i].p, written[i].bytes, read[j].p, read[j].bytes))
                return true;
    }
    return false;
}

// Bytes of a matrix of `rows` rows, `stride` elements apart, `width` used in
// the last; false if that passes 2^62.
bool matrix_bytes(size_t rows, size_t stride, size_t width, size_t size, size_t *bytes)
{
    *bytes = 0;
    if (rows == 0 || width == 0) return true;
    const size_t most = (size_t(1) << 62) / size;
    if (stride != 0 && rows - 1 > (most - width) / stride) return false;
    *bytes = ((rows - 1) * stride + width) * size;
    return true;
}

// What the three block table calls check alike.
devscan_status paged_check(const void *table, size_t stride, size_t rows, int width, int page, size_t *table_bytes)
{
    if (width < 0 || page < 1 || rows >= static_cast<size_t>(INT32_MAX) || stride < static_cast<size_t>(width))
        return DEVSCAN_ERR_INVALID;
    if (!matrix_bytes(rows, stride, static_cast<size_t>(width), 4, table_bytes)) return DEVSCAN_ERR_INVALID;
    if (*table_bytes > 0 && (table == nullptr || misaligned(table, 4))) return DEVSCAN_ERR_INVALID;
    return DEVSCAN_OK;
}

// The workspace, and scratch for the scanned ends where they do not fit in a
// block's shared memory.
devscan_status paged_scratch(size_t rows, cudaStream_t stream, Workspace *ws, Hold *hold, int32_t **scratch)
{
    *scratch = nullptr;
    const devscan_status st = acquire(stream, 1, ws, hold);
    if (st != DEVSCAN_OK || rows <= static_cast<size_t>(kPagedSharedRows)) return st;
    void *p = nullptr;
    const devscan_status got = acquire_extra(stream, 2 * rows * sizeof(int32_t), &p);
    *scratch = static_cast<int32_t *>(p);
    return got;
}

// `call` as the caller gave it, vocab in `vocab`; logits of `size` bytes each.
devscan_status sample_common(cudaError_t (*launch)(const SampleCall &, const Workspace &, cudaStream_t), size_t size,
                             SampleCall call, size_t vocab, cudaStream_t stream)
{
    const size_t rows = call.rows;
    if (rows > static_cast<size_t>(INT32_MAX)) return DEVSCAN_ERR_INVALID;
    if (vocab < 1 || vocab > DEVSCAN_SAMPLE_MAX_VOCAB || call.stride < vocab) return DEVSCAN_ERR_INVALID;
    if (call.noise != nullptr && call.noise_stride < vocab) return DEVSCAN_ERR_INVALID;
    if (rows == 0) return DEVSCAN_OK;
    if (call.logits == nullptr || call.tokens == nullptr) return DEVSCAN_ERR_INVALID;
    if (misaligned(call.logits, size) || misaligned(call.noise, 4) || misaligned(call.temperature, 4) ||
        misaligned(call.top_k, 4) || misaligned(call.top_p, 4) || misaligned(call.min_p, 4) ||
        misaligned(call.tokens, 4) || misaligned(call.logprobs, 4))
        return DEVSCAN_ERR_INVALID;
    size_t x_bytes = 0, q_bytes = 0;
    if (!matrix_bytes(rows, call.stride, vocab, size, &x_bytes)) return DEVSCAN_ERR_INVALID;
    if (call.noise != nullptr && !matrix_bytes(rows, call.noise_stride, vocab, 4, &q_bytes))
        return DEVSCAN_ERR_INVALID;
    const size_t each = rows * 4;
    const Span written[] = {{call.tokens, each}, {call.logprobs, each}};
    const Span read[] = {{call.logits, x_bytes}, {call.noise, q_bytes}, {call.temperature, each},
                         {call.top_k, each},     {call.top_p, each},    {call.min_p, each}};
    if (written_overlap(written, read)) return DEVSCAN_ERR_INVALID;
    call.vocab = static_cast<unsigned>(vocab);
    Workspace ws;
    Hold hold;
    devscan_status st = acquire(stream, 1, &ws, &hold);
    if (st != DEVSCAN_OK) return st;
    if (call.noise != nullptr && (call.top_k != nullptr || call.top_p != nullptr)) {
        void *row_words = nullptr;
        st = acquire_extra(stream, rows * sizeof(uint32_t), &row_words);
        if (st != DEVSCAN_OK) return st;
        call.row_words = static_cast<uint32_t *>(row_words);
    }
    return from_cuda(launch(call, ws, stream));
}

// A call's array of values: rows of tokens of neighbouring channels, strides
// in elements of `size` bytes.
struct Values {
    GatedArray array;
    size_t size;
    size_t bytes;   // from the first to behind the last
};

// Fills `bytes`; false where an argument is no good.  An output's tokens must
// not overlap each other.
bool check_values(Values *v, const GatedRows &rows, bool output)
{
    const size_t r = rows.starts != nullptr ? 1 : static_cast<size_t>(rows.rows), t = rows.tokens;
    const size_t c = static_cast<size_t>(rows.channels);
    v->bytes = 0;
    if (r == 0 || t == 0) return true;
    if (v->array.data == nullptr || misaligned(v->array.data, v->size)) return false;
    const size_t most = (size_t(1) << 61) / v->size;
    size_t rs = r > 1 ? v->array.row_stride : 0, ts = t > 1 ? v->array.stride : 0;
    if ((rs != 0 && r - 1 > most / rs) || (ts != 0 && t - 1 > most / ts) || c > most) return false;
    if (output) {
        const bool rows_apart = r == 1 || rs >= (t - 1) * ts + c, tokens_apart = t == 1 || ts >= (r - 1) * rs + c;
        if ((t > 1 && ts < c) || (r > 1 && rs < c) || !(rows_apart || tokens_apart)) return false;
    }
    v->bytes = ((r - 1) * rs + (t - 1) * ts + c) * v->size;
    return true;
}

// Whether an output and another array may share memory: not where they lie
// apart, nor where both have the same strides and their channels lie side by
// side within a token's: every token begins at a multiple of the strides'
// common divisor, and modulo that the two are apart.  (Batch-major tokens are
// their own stride apart, time-major ones their rows'.)
bool values_overlap(const Values &a, const Values &b, const GatedRows &rows)
{
    if (a.bytes == 0 || b.bytes == 0 || !overlaps(a.array.data, a.bytes, b.array.data, b.bytes)) return false;
    const bool one_row = rows.starts != nullptr || rows.rows == 1, one_token = rows.tokens == 1;
    if (one_row && one_token) return true;
    const size_t row = one_row ? 0 : a.array.row_stride * a.size, row_b = one_row ? 0 : b.array.row_stride * b.size;
    const size_t step = one_token ? 0 : a.array.stride * a.size, step_b = one_token ? 0 : b.array.stride * b.size;
    const size_t apart = std::gcd(row, step);
    if (apart == 0 || row != row_b || step != step_b) return true;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.array.data), y = reinterpret_cast<uintptr_t>(b.array.data);
    const size_t shift = x <= y ? (y - x) % apart : (apart - (x - y) % apart) % apart;   // of b within a's token
    const size_t c = static_cast<size_t>(rows.channels);
    return shift < c * a.size || shift + c * b.size > apart;
}

// What forward and backward check alike.
devscan_status gated_check(size_t rows, size_t tokens, size_t channels, const int32_t *starts, const int32_t *slots,
                           size_t pool, devscan_gate kind, GatedRows *out)
{
    if (kind != DEVSCAN_GATE_DECAY && kind != DEVSCAN_GATE_LOG && kind != DEVSCAN_GATE_SIGMOID)
        return DEVSCAN_ERR_INVALID;
    constexpr size_t kMost = static_cast<size_t>(INT32_MAX) - 1;
    constexpr size_t kMostChannels = kMost - 128;   // the last lanes of the last warp are counted too
    if (rows > kMost || tokens > kMost || channels > kMostChannels || pool > kMost || channels < 1) return DEVSCAN_ERR_INVALID;
    if (starts == nullptr && rows * tokens > kMost) return DEVSCAN_ERR_INVALID;
    if (misaligned(starts, 4) || misaligned(slots, 4)) return DEVSCAN_ERR_INVALID;
    *out = {starts, slots, static_cast<int>(rows), static_cast<int>(channels), static_cast<int>(pool),
            static_cast<unsigned>(tokens), 0, 0, 0, 0};
    return DEVSCAN_OK;
}

devscan_status current_sms(int *sms)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return DEVSCAN_ERR_CUDA;
    return DEVSCAN_OK;
}

using GatedScanLaunch = cudaError_t (*)(const GatedScanCall &, bool, int, cudaStream_t);
using GatedBackwardLaunch = cudaError_t (*)(const GatedBackwardCall &, bool, int, cudaStream_t);

devscan_status gated_scan_common(GatedScanLaunch launch, size_t size, GatedScanCall call, int gate_f32, size_t rows,
                                 size_t tokens, size_t channels, size_t pool, devscan_gate kind, cudaStream_t stream)
{
    devscan_status st = gated_check(rows, tokens, channels, call.rows.starts, call.rows.slots, pool, kind, &call.rows);
    if (st != DEVSCAN_OK) return st;
    call.kind = kind;
    if (rows == 0 && call.rows.starts == nullptr) return DEVSCAN_OK;
    const bool wide = size == 2 && gate_f32 != 0;
    Values x = {call.x, size, 0}, gate = {call.gate, wide ? 4 : size, 0}, out = {call.out, size, 0};
    if (!check_values(&x, call.rows, false) || !check_values(&gate, call.rows, false) || !check_values(&out, call.rows, true))
        return DEVSCAN_ERR_INVALID;
    if (misaligned(call.initial, 4) || misaligned(call.final, 4)) return DEVSCAN_ERR_INVALID;
    if (call.rows.slots == nullptr && (call.initial != nullptr || call.final != nullptr) && pool < rows)
        return DEVSCAN_ERR_INVALID;
    size_t states = 0;
    if (!matrix_bytes(pool, channels, channels, 4, &states)) return DEVSCAN_ERR_INVALID;
    const bool in_place = out.array.data == x.array.data && out.array.stride == x.array.stride &&
                          out.array.row_stride == x.array.row_stride;
    if ((!in_place && values_overlap(out, x, call.rows)) || values_overlap(out, gate, call.rows)) return DEVSCAN_ERR_INVALID;
    const size_t starts = call.rows.starts != nullptr ? (rows + 1) * 4 : 0, slots = rows * 4;
    const Span written[] = {{out.array.data, out.bytes}, {call.final, states}};
    const Span read[] = {{call.rows.starts, starts}, {call.rows.slots, slots}};
    if (written_overlap(written, read)) return DEVSCAN_ERR_INVALID;
    if (call.initial != call.final) {   // the states in place are the same pool
        const Span next[] = {{call.final, states}}, last[] = {{call.initial, states}};
        if (written_overlap(next, last)) return DEVSCAN_ERR_INVALID;
    }
    const Span result[] = {{out.array.data, out.bytes}}, before[] = {{call.initial, states}};
    const Span next[] = {{call.final, states}}, values[] = {{x.array.data, x.bytes}, {gate.array.data, gate.bytes}};
    if (written_overlap(result, before) || written_overlap(next, values)) return DEVSCAN_ERR_INVALID;
    int sms = 0;
    st = current_sms(&sms);
    return st != DEVSCAN_OK ? st : from_cuda(launch(call, wide, sms, stream));
}

devscan_status gated_backward_common(GatedBackwardLaunch launch, size_t size, GatedBackwardCall call, int gate_f32,
                                     size_t rows, size_t tokens, size_t channels, devscan_gate kind, cudaStream_t stream)
{
    devscan_status st = gated_check(rows, tokens, channels, call.rows.starts, nullptr, rows, kind, &call.rows);
    if (st != DEVSCAN_OK) return st;
    call.kind = kind;
    if (rows == 0 && call.rows.starts == nullptr) return DEVSCAN_OK;
    const bool wide = size == 2 && gate_f32 != 0, sigmoid = kind == DEVSCAN_GATE_SIGMOID;
    const size_t gate_size = wide ? 4 : size;
    Values in[] = {{call.grad, size, 0}, {call.gate, gate_size, 0}, {call.y, size, 0}, {call.x, size, 0}};
    Values out[] = {{call.grad_x, size, 0}, {call.grad_gate, gate_size, 0}};
    const int ins = sigmoid ? 4 : 3;
    for (int i = 0; i < ins; ++i)
        if (!check_values(&in[i], call.rows, false)) return DEVSCAN_ERR_INVALID;
    for (Values &v : out)
        if (!check_values(&v, call.rows, true)) return DEVSCAN_ERR_INVALID;
    if (misaligned(call.initial, 4) || misaligned(call.grad_final, 4) || misaligned(call.grad_initial, 4))
        return DEVSCAN_ERR_INVALID;
    for (const Values &v : out)
        for (int i = 0; i < ins; ++i)
            if (values_overlap(v, in[i], call.rows)) return DEVSCAN_ERR_INVALID;
    if (values_overlap(out[0], out[1], call.rows)) return DEVSCAN_ERR_INVALID;
    size_t states = 0;
    if (!matrix_bytes(rows, channels, channels, 4, &states)) return DEVSCAN_ERR_INVALID;
    const size_t starts = call.rows.starts != nullptr ? (rows + 1) * 4 : 0;
    const Span more[] = {{call.rows.starts, starts}, {call.initial, states}, {call.grad_final, states}};
    for (const Values &v : out) {
        const Span written[] = {{v.array.data, v.bytes}, {call.grad_initial, states}};
        if (written_overlap(written, more)) return DEVSCAN_ERR_INVALID;
    }
    for (int i = 0; i < ins; ++i) {
        const Span written[] = {{call.grad_initial, states}}, read[] = {{in[i].array.data, in[i].bytes}};
        if (written_overlap(written, read)) return DEVSCAN_ERR_INVALID;
    }
    int sms = 0;
    st = current_sms(&sms);
    return st != DEVSCAN_OK ? st : from_cuda(launch(call, wide, sms, stream));
}

devscan_status expert_sort_common(const void *ids, size_t id_size, size_t tokens, size_t choices, size_t experts,
                                  size_t align, size_t rows, int32_t *starts, int32_t *counts, int32_t *order,
                                  int32_t *places, cudaStream_t stream)
{
    constexpr size_t kMost = INT32_MAX;
    if (experts < 1 || experts > static_cast<size_t>(kMostExperts) || align < 1 || choices < 1) return DEVSCAN_ERR_INVALID;
    if (tokens > kMost || choices > kMost || tokens * choices > kMost || rows > kMost || align > kMost)
        return DEVSCAN_ERR_INVALID;
    const size_t pairs = tokens * choices;
    if (pairs + experts * (align - 1) > kMost) return DEVSCAN_ERR_INVALID;
    if (starts == nullptr || counts == nullptr || (rows > 0 && order == nullptr) ||
        (pairs > 0 && (ids == nullptr || places == nullptr)))
        return DEVSCAN_ERR_INVALID;
    if (misaligned(ids, id_size) || misaligned(starts, 4) || misaligned(counts, 4) || misaligned(order, 4) ||
        misaligned(places, 4))
        return DEVSCAN_ERR_INVALID;
    const Span written[] = {{starts, (experts + 1) * 4}, {counts, experts * 4}, {order, rows * 4}, {places, pairs * 4}};
    const Span read[] = {{ids, pairs * id_size}};
    if (written_overlap(written, read)) return DEVSCAN_ERR_INVALID;
    return from_cuda(launch_expert_sort({ids, static_cast<unsigned>(pairs), static_cast<unsigned>(rows),
                                         static_cast<unsigned>(align), static_cast<int>(experts), starts, counts, order,
                                         places, false},
                                        id_size == 8, stream));
}

// What the calls on rows of experts check alike: sizes, and the places.
bool expert_sizes(size_t tokens, size_t choices, size_t rows, size_t width)
{
    constexpr size_t kMost = INT32_MAX;
    return choices >= 1 && width >= 1 && tokens <= kMost && choices <= kMost && rows <= kMost && width <= kMost &&
           tokens * choices <= kMost;
}

// More tokens and rows than a grid has blocks are an argument's fault.
devscan_status from_grid(cudaError_t e) { return e == cudaErrorInvalidConfiguration ? DEVSCAN_ERR_INVALID : from_cuda(e); }

devscan_status expert_combine_common(ValueType type, const ExpertCombineCall &call, size_t rows, size_t tokens,
                                     size_t choices, size_t width, cudaStream_t stream)
{
    const size_t size = type == ValueType::F32 ? 4 : 2;
    if (!expert_sizes(tokens, choices, rows, width)) return DEVSCAN_ERR_INVALID;
    if ((rows > 1 && call.y_stride < width) || (tokens > 1 && call.out_stride < width)) return DEVSCAN_ERR_INVALID;
    if (tokens == 0) return DEVSCAN_OK;
    if (call.places == nullptr || call.out == nullptr || (rows > 0 && call.y == nullptr)) return DEVSCAN_ERR_INVALID;
    if (misaligned(call.y, size) || misaligned(call.out, size) || misaligned(call.places, 4) || misaligned(call.weights, 4))
        return DEVSCAN_ERR_INVALID;
    size_t y_bytes = 0, out_bytes = 0;
    if (!matrix_bytes(rows, call.y_stride, width, size, &y_bytes) ||
        !matrix_bytes(tokens, call.out_stride, width, size, &out_bytes))
        return DEVSCAN_ERR_INVALID;
    const Span written[] = {{call.out, out_bytes}};
    const Span read[] = {{call.y, y_bytes}, {call.places, tokens * choices * 4}, {call.weights, tokens * choices * 4}};
    if (written_overlap(written, read)) return DEVSCAN_ERR_INVALID;
    ExpertCombineCall c = call;
    c.rows = static_cast<unsigned>(rows), c.tokens = static_cast<unsigned>(tokens);
    c.width = static_cast<unsigned>(width), c.choices = static_cast<int>(choices);
    return from_grid(launch_expert_combine(type, c, stream));
}

devscan_status expert_combine_backward_common(ValueType type, const ExpertCombineBackwardCall &call, size_t rows,
                                              size_t tokens, size_t choices, size_t width, cudaStream_t stream)
{
    const size_t size = type == ValueType::F32 ? 4 : 2;
    if (!expert_sizes(tokens, choices, rows, width)) return DEVSCAN_ERR_INVALID;
    if ((rows > 1 && (call.y_stride < width || call.grad_y_stride < width)) || (tokens > 1 && call.grad_stride < width))
        return DEVSCAN_ERR_INVALID;
    if (tokens > 0 && (call.places == nullptr || call.grad == nullptr)) return DEVSCAN_ERR_INVALID;
    if (rows > 0 && (call.grad_y == nullptr || (call.grad_weights != nullptr && call.y == nullptr)))
        return DEVSCAN_ERR_INVALID;
    if (misaligned(call.grad, size) || misaligned(call.y, size) || misaligned(call.grad_y, size) ||
        misaligned(call.places, 4) || misaligned(call.order, 4) || misaligned(call.weights, 4) ||
        misaligned(call.grad_weights, 4))
        return DEVSCAN_ERR_INVALID;
    size_t grad_bytes = 0, y_bytes = 0, grad_y_bytes = 0;
    if (!matrix_bytes(tokens, call.grad_stride, width, size, &grad_bytes) ||
        !matrix_bytes(rows, call.y_stride, width, size, &y_bytes) ||
        !matrix_bytes(rows, call.grad_y_stride, width, size, &grad_y_bytes))
        return DEVSCAN_ERR_INVALID;
    const size_t pairs = tokens * choices * 4;
    const Span written[] = {{call.grad_y, grad_y_bytes}, {call.grad_weights, pairs}};
    const Span read[] = {{call.grad, grad_bytes}, {call.y, y_bytes},   {call.places, pairs},
                         {call.order, rows * 4},  {call.weights, pairs}};
    if (written_overlap(written, read)) return DEVSCAN_ERR_INVALID;
    ExpertCombineBackwardCall c = call;
    c.rows = static_cast<unsigned>(rows), c.tokens = static_cast<unsigned>(tokens);
    c.width = static_cast<unsigned>(width), c.choices = static_cast<int>(choices);
    return from_grid(launch_expert_combine_backward(type, c, stream));
}

devscan_status norm_common(const devscan_tensor *tensors, size_t count, bool clip, float max_norm, float *norm, void *work,
                           size_t work_bytes, cudaStream_t stream)
try {
    static_assert(DEVSCAN_NORM_WORK_TENSORS == kNormTensors && DEVSCAN_NORM_WORK_BYTES(1) == kNormBlocks * sizeof(double),
                  "the header's scratch is the launch's");
    constexpr size_t kMostTensors = size_t(1) << 24;
    if (norm == nullptr || misaligned(norm, 4) || work == nullptr || misaligned(work, 8)) return DEVSCAN_ERR_INVALID;
    if (count > kMostTensors || (count > 0 && tensors == nullptr)) return DEVSCAN_ERR_INVALID;
    if (clip && !(max_norm >= 0.0f)) return DEVSCAN_ERR_INVALID;
    const size_t need = DEVSCAN_NORM_WORK_BYTES(count);
    if (work_bytes < need) return DEVSCAN_ERR_INVALID;
    const Span written[] = {{norm, 4}, {work, need}};
    std::vector<NormTensor> list(count);
    for (size_t i = 0; i < count; ++i) {
        const devscan_tensor &t = tensors[i];
        if (t.type != DEVSCAN_TYPE_F32 && t.type != DEVSCAN_TYPE_F16 && t.type != DEVSCAN_TYPE_BF16)
            return DEVSCAN_ERR_INVALID;
        const size_t size = t.type == DEVSCAN_TYPE_F32 ? 4 : 2;
        if (t.n > (size_t(1) << 60)) return DEVSCAN_ERR_INVALID;
        list[i] = {t.in, clip ? t.out : nullptr, t.n, static_cast<ValueType>(t.type)};
        if (t.n == 0) continue;
        if (t.in == nullptr || misaligned(t.in, size)) return DEVSCAN_ERR_INVALID;
        const Span in[] = {{t.in, t.n * size}};
        if (written_overlap(written, in)) return DEVSCAN_ERR_INVALID;
        if (!clip) continue;
        if (t.out == nullptr || misaligned(t.out, size)) return DEVSCAN_ERR_INVALID;
        const Span out[] = {{t.out, t.n * size}}, others[] = {{norm, 4}, {work, need}};
        if (written_overlap(out, others) || (t.out != t.in && written_overlap(out, in))) return DEVSCAN_ERR_INVALID;
    }
    int sms = 0, dev = 0;
    const devscan_status st = current_sms(&sms);
    if (st != DEVSCAN_OK) return st;
    if (cudaGetDevice(&dev) != cudaSuccess) return DEVSCAN_ERR_CUDA;
    // The second launch starts beside the first and reads the tensors, so no other
    // call's launch may come between them.
    Hold hold;
    hold_slot({dev, reinterpret_cast<uintptr_t>(stream)}, true, &hold);
    return from_cuda(launch_grad_norm(list.data(), count, clip, max_norm, norm, static_cast<double *>(work), sms, stream));
} catch (const std::bad_alloc &) {
    return DEVSCAN_ERR_NOMEM;
}

}  // namespace
}  // namespace devscan

using namespace devscan;

extern "C" {

devscan_status scan_inclusive_i32(const int32_t *in, int32_t *out, size_t n, devscan_op op, cudaStream_t stream)
{
    return scan_common(ElemType::I32, true, in, out, n, op, stream);
}
devscan_status scan_inclusive_u32(const uint32_t *in, uint32_t *out, size_t n, devscan_op op, cudaStream_t stream)
{
    return scan_common(ElemType::U32, true, in, out, n, op, stream);
}
devscan_status scan_inclusive_f32(const float *in, float *out, size_t n, devscan_op op, cudaStream_t stream)
{
    return scan_common(ElemType::F32, true, in, out, n, op, stream);
}
devscan_status scan_exclusive_i32(const int32_t *in, int32_t *out, size_t n, devscan_op op, cudaStream_t stream)
{
    return scan_common(ElemType::I32, false, in, out, n, op, stream);
}
devscan_status scan_exclusive_u32(const uint32_t *in, uint32_t *out, size_t n, devscan_op op, cudaStream_t stream)
{
    return scan_common(ElemType::U32, false, in, out, n, op, stream);
}
devscan_status scan_exclusive_f32(const float *in, float *out, size_t n, devscan_op op, cudaStream_t stream)
{
    return scan_common(ElemType::F32, false, in, out, n, op, stream);
}

devscan_status scan_inclusive_carry_i32(const int32_t *in, int32_t *out, size_t n, devscan_op op,
                                        const int32_t *carry_in, cudaStream_t stream)
{
    return scan_common(ElemType::I32, true, in, out, n, op, stream, carry_in);
}
devscan_status scan_inclusive_carry_u32(const uint32_t *in, uint32_t *out, size_t n, devscan_op op,
                                        const uint32_t *carry_in, cudaStream_t stream)
{
    return scan_common(ElemType::U32, true, in, out, n, op, stream, carry_in);
}
devscan_status scan_inclusive_carry_f32(const float *in, float *out, size_t n, devscan_op op, const float *carry_in,
                                        cudaStream_t stream)
{
    return scan_common(ElemType::F32, true, in, out, n, op, stream, carry_in);
}
devscan_status scan_exclusive_carry_i32(const int32_t *in, int32_t *out, size_t n, devscan_op op,
                                        const int32_t *carry_in, cudaStream_t stream)
{
    return scan_common(ElemType::I32, false, in, out, n, op, stream, carry_in);
}
devscan_status scan_exclusive_carry_u32(const uint32_t *in, uint32_t *out, size_t n, devscan_op op,
                                        const uint32_t *carry_in, cudaStream_t stream)
{
    return scan_common(ElemType::U32, false, in, out, n, op, stream, carry_in);
}
devscan_status scan_exclusive_carry_f32(const float *in, float *out, size_t n, devscan_op op, const float *carry_in,
                                        cudaStream_t stream)
{
    return scan_common(ElemType::F32, false, in, out, n, op, stream, carry_in);
}

devscan_status scan_inclusive_host_i32(const int32_t *h_in, int32_t *h_out, size_t n, devscan_op op, int32_t *d_in,
                                       int32_t *d_out, cudaStream_t stream)
{
    return scan_host_common(ElemType::I32, true, h_in, h_out, n, op, d_in, d_out, stream);
}
devscan_status scan_inclusive_host_u32(const uint32_t *h_in, uint32_t *h_out, size_t n, devscan_op op,
                                       uint32_t *d_in, uint32_t *d_out, cudaStream_t stream)
{
    return scan_host_common(ElemType::U32, true, h_in, h_out, n, op, d_in, d_out, stream);
}
devscan_status scan_inclusive_host_f32(const float *h_in, float *h_out, size_t n, devscan_op op, float *d_in,
                                       float *d_out, cudaStream_t stream)
{
    return scan_host_common(ElemType::F32, true, h_in, h_out, n, op, d_in, d_out, stream);
}
devscan_status scan_exclusive_host_i32(const int32_t *h_in, int32_t *h_out, size_t n, devscan_op op, int32_t *d_in,
                                       int32_t *d_out, cudaStream_t stream)
{
    return scan_host_common(ElemType::I32, false, h_in, h_out, n, op, d_in, d_out, stream);
}
devscan_status scan_exclusive_host_u32(const uint32_t *h_in, uint32_t *h_out, size_t n, devscan_op op,
                                       uint32_t *d_in, uint32_t *d_out, cudaStream_t stream)
{
    return scan_host_common(ElemType::U32, false, h_in, h_out, n, op, d_in, d_out, stream);
}
devscan_status scan_exclusive_host_f32(const float *h_in, float *h_out, size_t n, devscan_op op, float *d_in,
                                       float *d_out, cudaStream_t stream)
{
    return scan_host_common(ElemType::F32, false, h_in, h_out, n, op, d_in, d_out, stream);
}

devscan_status reduce_i32(const int32_t *in, size_t n, devscan_op op, int32_t *total, cudaStream_t stream)
{
    return reduce_common(ElemType::I32, in, n, op, total, stream);
}
devscan_status reduce_u32(const uint32_t *in, size_t n, devscan_op op, uint32_t *total, cudaStream_t stream)
{
    return reduce_common(ElemType::U32, in, n, op, total, stream);
}
devscan_status reduce_f32(const float *in, size_t n, devscan_op op, float *total, cudaStream_t stream)
{
    return reduce_common(ElemType::F32, in, n, op, total, stream);
}

devscan_status segmented_scan_inclusive_i32(const int32_t *in, const uint8_t *heads, int32_t *out, size_t n,
                                            devscan_op op, cudaStream_t stream)
{
    return segscan_common(ElemType::I32, true, in, heads, out, n, op, stream);
}
devscan_status segmented_scan_inclusive_u32(const uint32_t *in, const uint8_t *heads, uint32_t *out, size_t n,
                                            devscan_op op, cudaStream_t stream)
{
    return segscan_common(ElemType::U32, true, in, heads, out, n, op, stream);
}
devscan_status segmented_scan_inclusive_f32(const float *in, const uint8_t *heads, float *out, size_t n,
                                            devscan_op op, cudaStream_t stream)
{
    return segscan_common(ElemType::F32, true, in, heads, out, n, op, stream);
}
devscan_status segmented_scan_exclusive_i32(const int32_t *in, const uint8_t *heads, int32_t *out, size_t n,
                                            devscan_op op, cudaStream_t stream)
{
    return segscan_common(ElemType::I32, false, in, heads, out, n, op, stream);
}
devscan_status segmented_scan_exclusive_u32(const uint32_t *in, const uint8_t *heads, uint32_t *out, size_t n,
                                            devscan_op op, cudaStream_t stream)
{
    return segscan_common(ElemType::U32, false, in, heads, out, n, op, stream);
}
devscan_status segmented_scan_exclusive_f32(const float *in, const uint8_t *heads, float *out, size_t n,
                                            devscan_op op, cudaStream_t stream)
{
    return segscan_common(ElemType::F32, false, in, heads, out, n, op, stream);
}

devscan_status compact_i32(const int32_t *in, const uint8_t *flags, int32_t *out, int32_t *count, size_t n,
                           cudaStream_t stream)
{
    if (count == nullptr) return DEVSCAN_ERR_INVALID;
    if (n > static_cast<size_t>(INT32_MAX)) return DEVSCAN_ERR_INVALID;
    if (n > 0) {
        if (in == nullptr || flags == nullptr || out == nullptr) return DEVSCAN_ERR_INVALID;
        if (reinterpret_cast<uintptr_t>(in) % 4 != 0 || reinterpret_cast<uintptr_t>(out) % 4 != 0 ||
            reinterpret_cast<uintptr_t>(count) % 4 != 0)
            return DEVSCAN_ERR_INVALID;
        if (overlaps(out, n * 4, in, n * 4) || overlaps(out, n * 4, flags, n) || overlaps(count, 4, out, n * 4) ||
            overlaps(count, 4, in, n * 4) || overlaps(count, 4, flags, n))
            return DEVSCAN_ERR_INVALID;
    }
    if (n == 0) return from_cuda(cudaMemsetAsync(count, 0, sizeof(int32_t), stream));
    const unsigned tiles = tiles_for(n, kCompactTile);
    Workspace ws;
    Hold hold;
    devscan_status st = acquire(stream, tiles, &ws, &hold);
    if (st != DEVSCAN_OK) return st;
    const int carry = carry_mode();
    void *part_words = nullptr;   // the two-launch path's part counts and offsets
    if (carry == kCarryL2Resident || (carry == kCarryDefault && n >= kCompactTwoPassMinN)) {
        st = acquire_extra(stream, compact_part_words(n) * sizeof(uint32_t), &part_words);
        if (st != DEVSCAN_OK) return st;
    }
    return from_cuda(launch_compact(in, flags, out, count, n, carry, ws, kSpinLimit, stream,
                                    static_cast<uint32_t *>(part_words)));
}

devscan_status compact_gt_i32(const int32_t *in, int32_t threshold, int32_t *out, int32_t *count, size_t n,
                              cudaStream_t stream)
{
    if (count == nullptr || reinterpret_cast<uintptr_t>(count) % 4 != 0) return DEVSCAN_ERR_INVALID;
    if (n > static_cast<size_t>(INT32_MAX)) return DEVSCAN_ERR_INVALID;
    if (n > 0) {
        if (in == nullptr || out == nullptr) return DEVSCAN_ERR_INVALID;
        if (reinterpret_cast<uintptr_t>(in) % 4 != 0 || reinterpret_cast<uintptr_t>(out) % 4 != 0)
            return DEVSCAN_ERR_INVALID;
        if (overlaps(out, n * 4, in, n * 4) || overlaps(count, 4, out, n * 4) || overlaps(count, 4, in, n * 4))
            return DEVSCAN_ERR_INVALID;
    }
    if (n == 0) return from_cuda(cudaMemsetAsync(count, 0, sizeof(int32_t), stream));
    Workspace ws;
    Hold hold;
    devscan_status st = acquire(stream, tiles_for(n, kCompactTile), &ws, &hold);
    if (st != DEVSCAN_OK) return st;
    const int carry = carry_mode();
    void *part_words = nullptr;   // the two-launch path's part masks, counts and offsets
    if (carry == kCarryL2Resident) {
        st = acquire_extra(stream, compact_part_words(n) * sizeof(uint32_t), &part_words);
        if (st != DEVSCAN_OK) return st;
    }
    return from_cuda(launch_compact_gt(in, threshold, out, count, n, carry, ws, kSpinLimit, stream,
                                       static_cast<uint32_t *>(part_words)));
}

devscan_status bracket_scan_i32(const int32_t *in, int32_t *out, int32_t *result, size_t n, cudaStream_t stream)
{
    if (result == nullptr || reinterpret_cast<uintptr_t>(result) % 4 != 0) return DEVSCAN_ERR_INVALID;
    if (n > kMaxScanN) return DEVSCAN_ERR_INVALID;
    if (n > 0) {
        if (in == nullptr || reinterpret_cast<uintptr_t>(in) % 4 != 0) return DEVSCAN_ERR_INVALID;
        if (out != nullptr && reinterpret_cast<uintptr_t>(out) % 4 != 0) return DEVSCAN_ERR_INVALID;
        if (overlaps(result, 8, in, n * 4) || (out != nullptr && overlaps(result, 8, out, n * 4)))
            return DEVSCAN_ERR_INVALID;
    }
    Workspace ws;
    Hold hold;
    if (n > 0) {
        const devscan_status st = acquire(stream, tiles_for(n, kScanTile), &ws, &hold);
        if (st != DEVSCAN_OK) return st;
    }
    return from_cuda(launch_bracket(in, out, result, n, carry_mode(), ws,
                                    kSpinLimit, stream));
}

devscan_status split_bit_u32(const uint32_t *keys, uint32_t *out, int bit, size_t n, cudaStream_t stream)
{
    if (bit < 0 || bit > 31) return DEVSCAN_ERR_INVALID;
    if (n > static_cast<size_t>(INT32_MAX)) return DEVSCAN_ERR_INVALID;
    if (n == 0) return DEVSCAN_OK;
    if (keys == nullptr || out == nullptr) return DEVSCAN_ERR_INVALID;
    if (reinterpret_cast<uintptr_t>(keys) % 4 != 0 || reinterpret_cast<uintptr_t>(out) % 4 != 0)
        return DEVSCAN_ERR_INVALID;
    if (overlaps(keys, n * 4, out, n * 4)) return DEVSCAN_ERR_INVALID;
    const unsigned tiles = tiles_for(n, kSplitTile);
    Workspace ws;
    Hold hold;
    devscan_status st = acquire(stream, tiles, &ws, &hold);
    if (st != DEVSCAN_OK) return st;
    unsigned *z = &ws.state->zeros[40];
    const int carry = carry_mode();
    if (reinterpret_cast<uintptr_t>(keys) % 16 == 0 &&
        (carry == kCarryL2Resident || (carry == kCarryDefault && n >= kSplitTwoPassMinN))) {
        void *part_words = nullptr;   // the parts' zero offsets
        st = acquire_extra(stream, split_part_words(n) * sizeof(uint32_t), &part_words);
        if (st != DEVSCAN_OK) return st;
        return from_cuda(launch_split_two_pass(keys, out, n, bit, z, static_cast<uint32_t *>(part_words), ws, stream));
    }
    if (cudaMemsetAsync(z, 0, sizeof(unsigned), stream) != cudaSuccess) return DEVSCAN_ERR_CUDA;
    cudaError_t e = launch_count_zeros(keys, n, bit, z, ws, stream);
    if (e != cudaSuccess) return DEVSCAN_ERR_CUDA;
    return from_cuda(launch_split(keys, out, n, bit, z, nullptr, carry, ws, kSpinLimit, stream));
}

devscan_status radix_sort_u32(uint32_t *keys, uint32_t *tmp, size_t n, cudaStream_t stream)
{
    if (n > static_cast<size_t>(INT32_MAX)) return DEVSCAN_ERR_INVALID;
    if (n == 0) return DEVSCAN_OK;
    if (keys == nullptr || tmp == nullptr) return DEVSCAN_ERR_INVALID;
    if (reinterpret_cast<uintptr_t>(keys) % 4 != 0 || reinterpret_cast<uintptr_t>(tmp) % 4 != 0)
        return DEVSCAN_ERR_INVALID;
    if (overlaps(keys, n * 4, tmp, n * 4)) return DEVSCAN_ERR_INVALID;
    const unsigned tiles = tiles_for(n, kSplitTile);
    Workspace ws;
    Hold hold;
    devscan_status st = acquire(stream, tiles, &ws, &hold);
    if (st != DEVSCAN_OK) return st;
    unsigned *z = ws.state->zeros;   // z[b] = zero count of bit b
    const int carry = carry_mode();
    if (reinterpret_cast<uintptr_t>(keys) % 16 == 0 && reinterpret_cast<uintptr_t>(tmp) % 16 == 0 &&
        (carry == kCarryL2Resident || (carry == kCarryDefault && n >= kSortTwoPassMinN))) {
        void *part_words = nullptr;   // the parts' offsets, then the next pass's part counts
        st = acquire_extra(stream, sort_part_words(n) * sizeof(uint32_t), &part_words);
        if (st != DEVSCAN_OK) return st;
        return from_cuda(launch_sort_two_pass(keys, tmp, n, &z[40], static_cast<uint32_t *>(part_words), ws, stream));
    }
    if (cudaMemsetAsync(z, 0, 33 * sizeof(unsigned), stream) != cudaSuccess) return DEVSCAN_ERR_CUDA;
    if (launch_count_zeros(keys, n, 0, &z[0], ws, stream) != cudaSuccess) return DEVSCAN_ERR_CUDA;
    uint32_t *src = keys, *dst = tmp;
    for (int bit = 0; bit < 32; ++bit) {
        unsigned *next = (bit < 31) ? &z[bit + 1] : nullptr;
        if (launch_split(src, dst, n, bit, &z[bit], next, carry, ws, kSpinLimit, stream) != cudaSuccess)
            return DEVSCAN_ERR_CUDA;
        std::swap(src, dst);
    }
    return DEVSCAN_OK;
}

devscan_status radix_sort_digits_u32(uint32_t *keys, uint32_t *tmp, size_t n, cudaStream_t stream)
{
    if (n > static_cast<size_t>(INT32_MAX)) return DEVSCAN_ERR_INVALID;
    if (n == 0) return DEVSCAN_OK;
    if (keys == nullptr || tmp == nullptr) return DEVSCAN_ERR_INVALID;
    if (reinterpret_cast<uintptr_t>(keys) % 4 != 0 || reinterpret_cast<uintptr_t>(tmp) % 4 != 0)
        return DEVSCAN_ERR_INVALID;
    if (overlaps(keys, n * 4, tmp, n * 4)) return DEVSCAN_ERR_INVALID;
    const size_t hist_words = radix_hist_words(n);
    Workspace ws;
    Hold hold;
    devscan_status st = acquire(stream, tiles_for(hist_words, kScanTile), &ws, &hold);
    if (st != DEVSCAN_OK) return st;
    void *hist = nullptr;
    st = acquire_extra(stream, hist_words * sizeof(uint32_t), &hist);
    if (st != DEVSCAN_OK) return st;
    uint32_t *src = keys, *dst = tmp;
    for (int pass = 0; pass < kRadixPasses; ++pass) {
        if (launch_radix_pass(src, dst, n, pass, static_cast<uint32_t *>(hist), ws, kSpinLimit, stream) != cudaSuccess)
            return DEVSCAN_ERR_CUDA;
        std::swap(src, dst);
    }
    return DEVSCAN_OK;
}

devscan_status block_table_extend_i32(int32_t *table, size_t stride, size_t rows, int width, const int32_t *cached,
                                      const int32_t *fresh, int page, const int32_t *pages, size_t pool,
                                      const int32_t *free, uint8_t *granted, int32_t *left, cudaStream_t stream)
{
    size_t table_bytes = 0;
    devscan_status st = paged_check(table, stride, rows, width, page, &table_bytes);
    if (st != DEVSCAN_OK) return st;
    if (pool >= static_cast<size_t>(INT32_MAX) || (pool > 0 && pages == nullptr)) return DEVSCAN_ERR_INVALID;
    if (free == nullptr || left == nullptr) return DEVSCAN_ERR_INVALID;
    if (rows > 0 && (cached == nullptr || fresh == nullptr || granted == nullptr)) return DEVSCAN_ERR_INVALID;
    if (misaligned(cached, 4) || misaligned(fresh, 4) || misaligned(pages, 4) || misaligned(free, 4) ||
        misaligned(left, 4))
        return DEVSCAN_ERR_INVALID;
    const Span written[] = {{table, table_bytes}, {granted, rows}, {left, 4}};
    const Span read[] = {{cached, rows * 4}, {fresh, rows * 4}, {pages, pool * 4}, {free, 4}};
    if (written_overlap(written, read)) return DEVSCAN_ERR_INVALID;
    Workspace ws;
    Hold hold;
    int32_t *scratch = nullptr;
    st = paged_scratch(rows, stream, &ws, &hold, &scratch);
    if (st != DEVSCAN_OK) return st;
    return from_cuda(launch_block_table_extend(table, stride, static_cast<int>(rows), width, cached, fresh, page,
                                               pages, static_cast<int>(pool), free, granted, left, scratch, ws,
                                               stream));
}

devscan_status slot_map_i32(const int32_t *table, size_t stride, size_t rows, int width, const int32_t *cached,
                            const int32_t *fresh, const uint8_t *granted, int page, size_t tokens, int32_t *starts,
                            int64_t *slots, int32_t *positions, int32_t *row_ids, cudaStream_t stream)
{
    size_t table_bytes = 0;
    devscan_status st = paged_check(table, stride, rows, width, page, &table_bytes);
    if (st != DEVSCAN_OK) return st;
    if (tokens > static_cast<size_t>(INT32_MAX) || starts == nullptr) return DEVSCAN_ERR_INVALID;
    if (rows > 0 && (cached == nullptr || fresh == nullptr)) return DEVSCAN_ERR_INVALID;
    if (tokens > 0 && (slots == nullptr || positions == nullptr || row_ids == nullptr)) return DEVSCAN_ERR_INVALID;
    if (misaligned(cached, 4) || misaligned(fresh, 4) || misaligned(starts, 4) || misaligned(slots, 8) ||
        misaligned(positions, 4) || misaligned(row_ids, 4))
        return DEVSCAN_ERR_INVALID;
    const Span written[] = {{starts, (rows + 1) * 4}, {slots, tokens * 8}, {positions, tokens * 4},
                            {row_ids, tokens * 4}};
    const Span read[] = {{table, table_bytes}, {cached, rows * 4}, {fresh, rows * 4}, {granted, rows}};
    if (written_overlap(written, read)) return DEVSCAN_ERR_INVALID;
    Workspace ws;
    Hold hold;
    int32_t *scratch = nullptr;
    st = paged_scratch(rows, stream, &ws, &hold, &scratch);
    if (st != DEVSCAN_OK) return st;
    return from_cuda(launch_slot_map(table, stride, static_cast<int>(rows), width, cached, fresh, granted, page,
                                     static_cast<int>(tokens), starts, slots, positions, row_ids, scratch, ws,
                                     stream));
}

devscan_status block_table_release_i32(const int32_t *table, size_t stride, size_t rows, int width,
                                       const int32_t *cached, const uint8_t *done, int page, int32_t *pages,
                                       size_t pool, const int32_t *free, int32_t *left, cudaStream_t stream)
{
    size_t table_bytes = 0;
    devscan_status st = paged_check(table, stride, rows, width, page, &table_bytes);
    if (st != DEVSCAN_OK) return st;
    if (pool >= static_cast<size_t>(INT32_MAX) || (pool > 0 && pages == nullptr)) return DEVSCAN_ERR_INVALID;
    if (free == nullptr || left == nullptr) return DEVSCAN_ERR_INVALID;
    if (rows > 0 && (cached == nullptr || done == nullptr)) return DEVSCAN_ERR_INVALID;
    if (misaligned(cached, 4) || misaligned(pages, 4) || misaligned(free, 4) || misaligned(left, 4))
        return DEVSCAN_ERR_INVALID;
    const Span written[] = {{pages, pool * 4}, {left, 4}};
    const Span read[] = {{table, table_bytes}, {cached, rows * 4}, {done, rows}, {free, 4}};
    if (written_overlap(written, read)) return DEVSCAN_ERR_INVALID;
    Workspace ws;
    Hold hold;
    int32_t *scratch = nullptr;
    st = paged_scratch(rows, stream, &ws, &hold, &scratch);
    if (st != DEVSCAN_OK) return st;
    return from_cuda(launch_block_table_release(table, stride, static_cast<int>(rows), width, cached, done, page,
                                                pages, static_cast<int>(pool), free, left, scratch, ws, stream));
}

devscan_status sample_tokens_f32(const float *logits, size_t rows, size_t vocab, size_t logits_stride,
                                 const float *noise, size_t noise_stride, const float *temperature,
                                 const int32_t *top_k, const float *top_p, const float *min_p, int32_t *tokens,
                                 float *logprobs, cudaStream_t stream)
{
    return sample_common(launch_sample_f32, 4,
                         {logits, rows, logits_stride, 0, noise, noise_stride, temperature, top_k, top_p, min_p, tokens,
                          logprobs, nullptr},
                         vocab, stream);
}
devscan_status sample_tokens_f16(const uint16_t *logits, size_t rows, size_t vocab, size_t logits_stride,
                                 const float *noise, size_t noise_stride, const float *temperature,
                                 const int32_t *top_k, const float *top_p, const float *min_p, int32_t *tokens,
                                 float *logprobs, cudaStream_t stream)
{
    return sample_common(launch_sample_f16, 2,
                         {logits, rows, logits_stride, 0, noise, noise_stride, temperature, top_k, top_p, min_p, tokens,
                          logprobs, nullptr},
                         vocab, stream);
}
devscan_status sample_tokens_bf16(const uint16_t *logits, size_t rows, size_t vocab, size_t logits_stride,
                                  const float *noise, size_t noise_stride, const float *temperature,
                                  const int32_t *top_k, const float *top_p, const float *min_p, int32_t *tokens,
                                  float *logprobs, cudaStream_t stream)
{
    return sample_common(launch_sample_bf16, 2,
                         {logits, rows, logits_stride, 0, noise, noise_stride, temperature, top_k, top_p, min_p, tokens,
                          logprobs, nullptr},
                         vocab, stream);
}

devscan_status gated_scan_f32(const float *x, size_t x_row_stride, size_t x_stride, const void *gate,
                             size_t gate_row_stride, size_t gate_stride, int gate_f32, size_t rows, size_t tokens,
                             size_t channels, const int32_t *starts, const float *initial, const int32_t *slots,
                             size_t pool, devscan_gate kind, float *out, size_t out_row_stride, size_t out_stride,
                             float *final, cudaStream_t stream)
{
    GatedScanCall call = {};
    call.rows.starts = starts, call.rows.slots = slots;
    call.x = {const_cast<float *>(x), x_row_stride, x_stride};
    call.gate = {const_cast<void *>(gate), gate_row_stride, gate_stride};
    call.out = {out, out_row_stride, out_stride};
    call.initial = const_cast<float *>(initial), call.final = final;
    return gated_scan_common(launch_gated_scan_f32, 4, call, gate_f32, rows, tokens, channels, pool, kind, stream);
}

devscan_status gated_scan_backward_f32(const float *grad, size_t grad_row_stride, size_t grad_stride, const float *x,
                                      size_t x_row_stride, size_t x_stride, const void *gate, size_t gate_row_stride,
                                      size_t gate_stride, int gate_f32, const float *y, size_t y_row_stride,
                                      size_t y_stride, size_t rows, size_t tokens, size_t channels,
                                      const int32_t *starts, const float *initial, const float *grad_final,
                                      devscan_gate kind, float *grad_x, size_t grad_x_row_stride, size_t grad_x_stride,
                                      void *grad_gate, size_t grad_gate_row_stride, size_t grad_gate_stride,
                                      float *grad_initial, cudaStream_t stream)
{
    GatedBackwardCall call = {};
    call.rows.starts = starts;
    call.grad = {const_cast<float *>(grad), grad_row_stride, grad_stride};
    call.x = {const_cast<float *>(x), x_row_stride, x_stride};
    call.gate = {const_cast<void *>(gate), gate_row_stride, gate_stride};
    call.y = {const_cast<float *>(y), y_row_stride, y_stride};
    call.grad_x = {grad_x, grad_x_row_stride, grad_x_stride};
    call.grad_gate = {grad_gate, grad_gate_row_stride, grad_gate_stride};
    call.initial = const_cast<float *>(initial), call.grad_final = grad_final, call.grad_initial = grad_initial;
    return gated_backward_common(launch_gated_backward_f32, 4, call, gate_f32, rows, tokens, channels, kind, stream);
}

devscan_status gated_scan_f16(const uint16_t *x, size_t x_row_stride, size_t x_stride, const void *gate,
                             size_t gate_row_stride, size_t gate_stride, int gate_f32, size_t rows, size_t tokens,
                             size_t channels, const int32_t *starts, const float *initial, const int32_t *slots,
                             size_t pool, devscan_gate kind, uint16_t *out, size_t out_row_stride, size_t out_stride,
                             float *final, cudaStream_t stream)
{
    GatedScanCall call = {};
    call.rows.starts = starts, call.rows.slots = slots;
    call.x = {const_cast<uint16_t *>(x), x_row_stride, x_stride};
    call.gate = {const_cast<void *>(gate), gate_row_stride, gate_stride};
    call.out = {out, out_row_stride, out_stride};
    call.initial = const_cast<float *>(initial), call.final = final;
    return gated_scan_common(launch_gated_scan_f16, 2, call, gate_f32, rows, tokens, channels, pool, kind, stream);
}

devscan_status gated_scan_backward_f16(const uint16_t *grad, size_t grad_row_stride, size_t grad_stride, const uint16_t *x,
                                      size_t x_row_stride, size_t x_stride, const void *gate, size_t gate_row_stride,
                                      size_t gate_stride, int gate_f32, const uint16_t *y, size_t y_row_stride,
                                      size_t y_stride, size_t rows, size_t tokens, size_t channels,
                                      const int32_t *starts, const float *initial, const float *grad_final,
                                      devscan_gate kind, uint16_t *grad_x, size_t grad_x_row_stride, size_t grad_x_stride,
                                      void *grad_gate, size_t grad_gate_row_stride, size_t grad_gate_stride,
                                      float *grad_initial, cudaStream_t stream)
{
    GatedBackwardCall call = {};
    call.rows.starts = starts;
    call.grad = {const_cast<uint16_t *>(grad), grad_row_stride, grad_stride};
    call.x = {const_cast<uint16_t *>(x), x_row_stride, x_stride};
    call.gate = {const_cast<void *>(gate), gate_row_stride, gate_stride};
    call.y = {const_cast<uint16_t *>(y), y_row_stride, y_stride};
    call.grad_x = {grad_x, grad_x_row_stride, grad_x_stride};
    call.grad_gate = {grad_gate, grad_gate_row_stride, grad_gate_stride};
    call.initial = const_cast<float *>(initial), call.grad_final = grad_final, call.grad_initial = grad_initial;
    return gated_backward_common(launch_gated_backward_f16, 2, call, gate_f32, rows, tokens, channels, kind, stream);
}

devscan_status gated_scan_bf16(const uint16_t *x, size_t x_row_stride, size_t x_stride, const void *gate,
                             size_t gate_row_stride, size_t gate_stride, int gate_f32, size_t rows, size_t tokens,
                             size_t channels, const int32_t *starts, const float *initial, const int32_t *slots,
                             size_t pool, devscan_gate kind, uint16_t *out, size_t out_row_stride, size_t out_stride,
                             float *final, cudaStream_t stream)
{
    GatedScanCall call = {};
    call.rows.starts = starts, call.rows.slots = slots;
    call.x = {const_cast<uint16_t *>(x), x_row_stride, x_stride};
    call.gate = {const_cast<void *>(gate), gate_row_stride, gate_stride};
    call.out = {out, out_row_stride, out_stride};
    call.initial = const_cast<float *>(initial), call.final = final;
    return gated_scan_common(launch_gated_scan_bf16, 2, call, gate_f32, rows, tokens, channels, pool, kind, stream);
}

devscan_status gated_scan_backward_bf16(const uint16_t *grad, size_t grad_row_stride, size_t grad_stride, const uint16_t *x,
                                      size_t x_row_stride, size_t x_stride, const void *gate, size_t gate_row_stride,
                                      size_t gate_stride, int gate_f32, const uint16_t *y, size_t y_row_stride,
                                      size_t y_stride, size_t rows, size_t tokens, size_t channels,
                                      const int32_t *starts, const float *initial, const float *grad_final,
                                      devscan_gate kind, uint16_t *grad_x, size_t grad_x_row_stride, size_t grad_x_stride,
                                      void *grad_gate, size_t grad_gate_row_stride, size_t grad_gate_stride,
                                      float *grad_initial, cudaStream_t stream)
{
    GatedBackwardCall call = {};
    call.rows.starts = starts;
    call.grad = {const_cast<uint16_t *>(grad), grad_row_stride, grad_stride};
    call.x = {const_cast<uint16_t *>(x), x_row_stride, x_stride};
    call.gate = {const_cast<void *>(gate), gate_row_stride, gate_stride};
    call.y = {const_cast<uint16_t *>(y), y_row_stride, y_stride};
    call.grad_x = {grad_x, grad_x_row_stride, grad_x_stride};
    call.grad_gate = {grad_gate, grad_gate_row_stride, grad_gate_stride};
    call.initial = const_cast<float *>(initial), call.grad_final = grad_final, call.grad_initial = grad_initial;
    return gated_backward_common(launch_gated_backward_bf16, 2, call, gate_f32, rows, tokens, channels, kind, stream);
}

devscan_status expert_sort_i32(const int32_t *ids, size_t tokens, size_t choices, size_t experts, size_t align,
                              size_t rows, int32_t *starts, int32_t *counts, int32_t *order, int32_t *places,
                              cudaStream_t stream)
{
    return expert_sort_common(ids, sizeof(int32_t), tokens, choices, experts, align, rows, starts, counts, order, places,
                              stream);
}

devscan_status expert_sort_i64(const int64_t *ids, size_t tokens, size_t choices, size_t experts, size_t align,
                              size_t rows, int32_t *starts, int32_t *counts, int32_t *order, int32_t *places,
                              cudaStream_t stream)
{
    return expert_sort_common(ids, sizeof(int64_t), tokens, choices, experts, align, rows, starts, counts, order, places,
                              stream);
}

devscan_status expert_dispatch(const void *x, size_t x_stride, size_t row_bytes, size_t tokens, size_t choices,
                               const int32_t *places, size_t rows, const int32_t *order, void *out, size_t out_stride,
                               cudaStream_t stream)
{
    if (!expert_sizes(tokens, choices, rows, row_bytes)) return DEVSCAN_ERR_INVALID;
    if ((tokens > 1 && x_stride < row_bytes) || (rows > 1 && out_stride < row_bytes)) return DEVSCAN_ERR_INVALID;
    if (rows == 0) return DEVSCAN_OK;
    if (out == nullptr || (tokens > 0 && (x == nullptr || places == nullptr))) return DEVSCAN_ERR_INVALID;
    if (misaligned(places, 4) || misaligned(order, 4)) return DEVSCAN_ERR_INVALID;
    size_t x_bytes = 0, out_bytes = 0;
    if (!matrix_bytes(tokens, x_stride, row_bytes, 1, &x_bytes) || !matrix_bytes(rows, out_stride, row_bytes, 1, &out_bytes))
        return DEVSCAN_ERR_INVALID;
    const Span written[] = {{out, out_bytes}};
    const Span read[] = {{x, x_bytes}, {places, tokens * choices * 4}, {order, rows * 4}};
    if (written_overlap(written, read)) return DEVSCAN_ERR_INVALID;
    return from_grid(launch_expert_dispatch({x, x_stride, row_bytes, static_cast<unsigned>(tokens),
                                             static_cast<unsigned>(rows), static_cast<int>(choices), places, order, out,
                                             out_stride},
                                            stream));
}

devscan_status expert_combine_f32(const float *y, size_t y_stride, size_t rows, size_t tokens, size_t choices,
                                 size_t width, const int32_t *places, const float *weights, float *out,
                                 size_t out_stride, cudaStream_t stream)
{
    return expert_combine_common(ValueType::F32, {y, y_stride, 0, 0, 0, 0, places, weights, out, out_stride}, rows, tokens,
                                 choices, width, stream);
}

devscan_status expert_combine_backward_f32(const float *grad, size_t grad_stride, const float *y, size_t y_stride,
                                          size_t rows, size_t tokens, size_t choices, size_t width,
                                          const int32_t *places, const float *weights, const int32_t *order,
                                          float *grad_y, size_t grad_y_stride, float *grad_weights, cudaStream_t stream)
{
    return expert_combine_backward_common(ValueType::F32,
                                          {grad, grad_stride, y, y_stride, 0, 0, 0, 0, places, order, weights, grad_y,
                                           grad_y_stride, grad_weights},
                                          rows, tokens, choices, width, stream);
}

devscan_status expert_combine_f16(const uint16_t *y, size_t y_stride, size_t rows, size_t tokens, size_t choices,
                                 size_t width, const int32_t *places, const float *weights, uint16_t *out,
                                 size_t out_stride, cudaStream_t stream)
{
    return expert_combine_common(ValueType::F16, {y, y_stride, 0, 0, 0, 0, places, weights, out, out_stride}, rows, tokens,
                                 choices, width, stream);
}

devscan_status expert_combine_backward_f16(const uint16_t *grad, size_t grad_stride, const uint16_t *y, size_t y_stride,
                                          size_t rows, size_t tokens, size_t choices, size_t width,
                                          const int32_t *places, const float *weights, const int32_t *order,
                                          uint16_t *grad_y, size_t grad_y_stride, float *grad_weights, cudaStream_t stream)
{
    return expert_combine_backward_common(ValueType::F16,
                                          {grad, grad_stride, y, y_stride, 0, 0, 0, 0, places, order, weights, grad_y,
                                           grad_y_stride, grad_weights},
                                          rows, tokens, choices, width, stream);
}

devscan_status expert_combine_bf16(const uint16_t *y, size_t y_stride, size_t rows, size_t tokens, size_t choices,
                                 size_t width, const int32_t *places, const float *weights, uint16_t *out,
                                 size_t out_stride, cudaStream_t stream)
{
    return expert_combine_common(ValueType::BF16, {y, y_stride, 0, 0, 0, 0, places, weights, out, out_stride}, rows, tokens,
                                 choices, width, stream);
}

devscan_status expert_combine_backward_bf16(const uint16_t *grad, size_t grad_stride, const uint16_t *y, size_t y_stride,
                                          size_t rows, size_t tokens, size_t choices, size_t width,
                                          const int32_t *places, const float *weights, const int32_t *order,
                                          uint16_t *grad_y, size_t grad_y_stride, float *grad_weights, cudaStream_t stream)
{
    return expert_combine_backward_common(ValueType::BF16,
                                          {grad, grad_stride, y, y_stride, 0, 0, 0, 0, places, order, weights, grad_y,
                                           grad_y_stride, grad_weights},
                                          rows, tokens, choices, width, stream);
}

devscan_status grad_norm(const devscan_tensor *tensors, size_t count, float *norm, void *work, size_t work_bytes,
                         cudaStream_t stream)
{
    return norm_common(tensors, count, false, 0.0f, norm, work, work_bytes, stream);
}

devscan_status clip_grad_norm(const devscan_tensor *tensors, size_t count, float max_norm, float *norm, void *work,
                              size_t work_bytes, cudaStream_t stream)
{
    return norm_common(tensors, count, true, max_norm, norm, work, work_bytes, stream);
}

devscan_status devscan_device_status(cudaStream_t stream)
{
    if (cudaStreamSynchronize(stream) != cudaSuccess) return DEVSCAN_ERR_CUDA;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return DEVSCAN_ERR_CUDA;
    Hold hold;
    const Slot *slot = hold_slot({dev, reinterpret_cast<uintptr_t>(stream)}, false, &hold);
    if (slot == nullptr || slot->base == nullptr) return DEVSCAN_OK;
    unsigned err = 0;
    if (cudaMemcpy(&err, &slot->ws.state->error, sizeof(unsigned), cudaMemcpyDeviceToHost) != cudaSuccess)
        return DEVSCAN_ERR_CUDA;
    // A launch that gave up may have left its tile counter, epoch and status
    // words half-way; the stream is idle now, so start the workspace afresh.
    if (err != 0 && cudaMemset(slot->base, 0, slot->bytes) != cudaSuccess) return DEVSCAN_ERR_CUDA;
    return (err & kErrTimeout) ? DEVSCAN_ERR_TIMEOUT : DEVSCAN_OK;
}

const char *devscan_status_string(devscan_status status)
{
    switch (status) {
    case DEVSCAN_OK: return "ok";
    case DEVSCAN_ERR_INVALID: return "invalid argument";
    case DEVSCAN_ERR_UNSUPPORTED: return "operator not supported for this element type";
    case DEVSCAN_ERR_CUDA: return "CUDA runtime error";
    case DEVSCAN_ERR_TIMEOUT: return "inter-block wait timed out on the device";
    case DEVSCAN_ERR_NOMEM: return "out of device memory for the workspace";
    }
    return "unknown status";
}

devscan_status devscan_stream_release(cudaStream_t stream)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return DEVSCAN_ERR_CUDA;
    const SlotKey key{dev, reinterpret_cast<uintptr_t>(stream)};
    Hold hold;
    const Slot *slot = hold_slot(key, false, &hold);
    if (slot == nullptr) return DEVSCAN_OK;
    void *base = slot->base;
    void *extra = slot->extra;
    {
        std::lock_guard<std::mutex> lock(g_mutex);
        g_slots.erase(key);
    }
    if (extra != nullptr && cudaFreeAsync(extra, stream) != cudaSuccess) return DEVSCAN_ERR_CUDA;
    return base == nullptr ? DEVSCAN_OK : from_cuda(cudaFreeAsync(base, stream));
}

devscan_status devscan_measure_set_carry_mode(int mode)
{
    if (mode != kCarryDefault && mode != kCarryLookback && mode != kCarryReduceThenScan && mode != kCarryPipelined &&
        mode != kCarryL2Resident)
        return DEVSCAN_ERR_INVALID;
    t_carry_mode = mode;
    return DEVSCAN_OK;
}

devscan_status devscan_selftest_stalled_wait(unsigned int spin_limit, cudaStream_t stream)
{
    if (spin_limit == 0) return DEVSCAN_ERR_INVALID;
    Workspace ws;
    Hold hold;
    const devscan_status st = acquire(stream, 1, &ws, &hold);
    if (st != DEVSCAN_OK) return st;
    return from_cuda(launch_stalled_wait(ws, spin_limit, stream));
}

}  // extern "C"
