// C ABI of the output layer's losses: handles that hold the sizes and the
// workspace, and the calls that check their arguments and launch the kernels.
#include "outloss.hpp"

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>
#include <vector>

#include "bufcheck.hpp"

namespace {

constexpr double kFloatMax = 3.4028234e38;
constexpr uint64_t kMaxTokens = 1ull << 22, kMaxHidden = 1ull << 16, kMaxVocab = 1ull << 24;
constexpr int kMaxTop = 1024;

// Logits of a piece of the tokens that the caller leaves to the handle: 1 GB of
// them.  Their gradients (2 bytes each in bf16) are kept for up to kPiecesKept
// pieces before the products with them, whose float32 sums over more than that go
// through memory: 8192 x 128000 logits of hidden size 4096 in four pieces took
// 20.7 ms with every piece's product added to a sum in memory.
constexpr uint64_t kPieceLogits = 1ull << 28;
constexpr uint64_t kPiecesKept = 4;

// Bytes of weights that are packed at a time where they are not read as they are:
// kPackBytes of float32 weights and of bf16 rows that are no multiple of 16 bytes;
// kStrayBytes where bf16 rows are, which are read as they are but in a caller's
// odd view of a larger matrix.  Such a view of 1 GB goes in four turns then: 512
// tokens of 4096 x 128000 take 2.31 ms with gradients and 1.57 in one; 200 MB of
// 2048 x 50001 are packed at once.
constexpr uint64_t kPackBytes = 1ull << 30, kStrayBytes = 1ull << 28;

// Blocks of 64 products that are summed in the tensor cores before float32 sums
// take over: of float32 inputs (six products a block), of bf16 inputs for logits
// and float32 results, and for bf16 results (whose rounding is 2^-8).  The tensor
// cores cut every sum off, always downwards, so the error grows with the run: with 1
// and 8 (3, where A has three planes) losses and float32 gradients are as far from 64
// bits as float32 products are (2 to 7e-7 relative); with 2 and 16 they are twice as
// far, and 515 tokens of 515 x 10007 float32 take 154 us instead of 173, 4096 of
// 2048 x 50001 bf16 1592 instead of 1633; with 4 for bf16 1739.  Sums of a million
// terms of one sign for a bf16 result were 0.65% low (1.5 of its steps) in one run; in runs of 256 blocks they are
// 0.01% low.  8192 tokens of 4096 x 128000 take 17.5 ms so and 17.3 in one run, other
// cases as long: from 128 to 512 blocks there is no difference beyond the noise.
constexpr uint32_t kFloatRun = 1, kExactRun = 8, kPlanesRun = 3, kLongRun = 256;

ar_status cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return AR_OK;
    cudaGetLastError();  // reported here: not once more by whoever looks at the thread's last error
    return e == cudaErrorMemoryAllocation ? AR_ERR_NOMEM : AR_ERR_CUDA;
}

bool float_normal(double x) { return x >= 1.17549436e-38 && x <= kFloatMax; }
bool float_dtype(ar_dtype d) { return d == AR_FLOAT32 || d == AR_BFLOAT16; }
int esize(ar_dtype d) { return d == AR_BFLOAT16 ? 2 : 4; }
uint64_t up(uint64_t x, uint64_t to) { return (x + to - 1) / to * to; }

// The workspace's parts: offsets of each in one allocation.
struct Layout {
    uint64_t rows = 0, pitch = 0;    // padded tokens, padded D
    uint64_t piece = 0, pieces = 0;  // tokens at a time
    uint64_t kept = 0;               // tokens whose logits' gradients are kept
    uint64_t pack = 0, part_room = 0, wide = 0, sum_pitch = 0;  // entries packed at a time, floats, padded V, ... D
    int planes = 1, list = 1;
    size_t status = 0, count = 0, factor = 0, row = 0, counted = 0, ids = 0, shares = 0, entropy = 0, logits = 0;
    size_t ticket = 0, sums = 0, bad = 0, stats = 0, loss = 0, hidden = 0, weight = 0, z = 0, grad = 0, part = 0, sum = 0;
    size_t bytes = 0;
    size_t add(uint64_t n) {
        const size_t at = bytes;
        bytes += up(n, 256);
        return at;
    }
};

ar_status make_layout(uint64_t tokens, uint64_t hidden, uint64_t vocab, ar_dtype dtype, int top, uint64_t piece,
                      int gradients, Layout& l) {
    if (hidden < 1 || vocab < 1 || top < 0 || (dtype != AR_INT32 && !float_dtype(dtype))) return AR_ERR_INVALID_ARG;
    if (!float_dtype(dtype) || tokens > kMaxTokens || hidden > kMaxHidden || vocab > kMaxVocab || top > kMaxTop ||
        tokens * static_cast<uint64_t>(std::max(1, top)) > (1ull << 31))
        return AR_ERR_UNSUPPORTED;
    const uint64_t tile = ar::kLossTile;
    l.planes = dtype == AR_BFLOAT16 ? 1 : ar::kMaxPlanes;
    l.list = std::max(1, top);
    l.rows = std::max(tile, up(tokens, tile));
    l.pitch = up(hidden, 8);
    l.wide = up(vocab, tile);
    l.sum_pitch = up(hidden, tile);
    if (!gradients) piece = l.rows;  // no logits are stored
    if (piece == 0) piece = std::max(tile, kPieceLogits / l.wide / tile * tile);
    piece = std::min(up(std::min(piece, l.rows), tile), l.rows);
    l.pieces = (l.rows + piece - 1) / piece;
    l.piece = up((l.rows + l.pieces - 1) / l.pieces, tile);  // as even as whole tiles allow
    l.pieces = (l.rows + l.piece - 1) / l.piece;
    l.kept = std::min(l.pieces, kPiecesKept) * l.piece;
    // calls of a few tokens pack none (Call::few)
    const uint64_t pack_bytes = tokens <= ar::kFewTokens ? 0 : l.planes == 1 && l.pitch == hidden ? kStrayBytes : kPackBytes;
    l.pack = std::min(l.wide, std::max(tile, pack_bytes / (2 * l.planes * l.pitch) / tile * tile));
    const uint64_t n = l.rows, k = n * l.list;
    l.status = l.add(4);
    l.count = l.add(4);
    l.ticket = l.add(4);
    l.sums = l.add(8 * (n / ar::kJoinRows));
    l.bad = l.add(4 * (n / ar::kJoinRows));
    l.factor = l.add(4);
    l.row = l.add(4 * n);
    l.counted = l.add(4 * n);
    l.entropy = l.add(4 * n);
    l.ids = l.add(4 * k);
    l.shares = l.add(4 * k);
    l.logits = l.add(4 * k);
    l.stats = l.add(8 * std::max(l.piece * (l.wide / ar::kStatColumns), ar::kFewTokens * (l.wide / ar::kFewColumns)));
    l.loss = l.add(4 * n);
    l.hidden = l.add(2 * l.planes * n * l.pitch);
    l.weight = l.add(2 * l.planes * l.pack * l.pitch);
    if (gradients) {
        l.z = l.add(4 * l.piece * l.wide);
        l.grad = l.add(2 * l.planes * l.kept * l.wide);
        // the kept tokens' gradient once (packed weights are summed up there), and eight
        // parts of each tile or one for each pair of SMs, up to eight for each pair
        const uint64_t pairs = ar::kLossSms / 2, tiles = std::max(l.kept, l.wide) / tile * (l.sum_pitch / tile);
        l.part_room = std::max(l.kept * l.sum_pitch, std::min(8 * pairs, std::max(8 * tiles, pairs + 4)) * tile * tile);
        l.part = l.add(4 * l.part_room);
        // float32 gradients of weights are summed where the caller wants them
        if (l.kept < l.rows && dtype == AR_BFLOAT16) l.sum = l.add(4 * l.wide * l.sum_pitch);
    }
    return AR_OK;
}

}  // namespace

struct ar_output_loss_s {
    int device = 0;
    uint64_t tokens = 0, hidden = 0, vocab = 0;
    ar_dtype dtype = AR_BFLOAT16;
    int top = 0;
    bool gradients = false;
    Layout l;
    char* dev = nullptr;
    template <class T>
    T* at(size_t offset) const {
        return reinterpret_cast<T*>(dev + offset);
    }
    ~ar_output_loss_s() {
        if (dev) cudaFree(dev);
    }
};

namespace {

// A caller's matrix of `rows` rows.
struct Matrix {
    const void* p;
    uint64_t rows, width, stride;
    int es;
    uint64_t bytes() const { return ar::matrix_bytes(rows, width, stride, static_cast<uint64_t>(es)); }
};

bool on_device(int device) {
    int now = -1;
    return cudaGetDevice(&now) == cudaSuccess && now == device;
}

// Inputs, which may overlap one another, and outputs, which may overlap nothing.
ar_status check_matrices(const std::vector<Matrix>& in, const std::vector<Matrix>& out, int device) {
    std::vector<Matrix> all(out);
    all.insert(all.end(), in.begin(), in.end());
    for (size_t i = 0; i < all.size(); ++i) {
        const Matrix& m = all[i];
        if (m.stride < m.width || m.stride > (1ull << 40) || m.bytes() == ar::kTooManyBytes) return AR_ERR_INVALID_ARG;
        if (m.bytes() == 0) continue;
        const uintptr_t a = reinterpret_cast<uintptr_t>(m.p);
        if (!a || a % m.es || a + m.bytes() < a) return AR_ERR_INVALID_ARG;
        for (size_t j = 0; j < i && j < out.size(); ++j) {
            const uintptr_t b = reinterpret_cast<uintptr_t>(all[j].p);
            if (all[j].bytes() && a < b + all[j].bytes() && b < a + m.bytes()) return AR_ERR_INVALID_ARG;
        }
    }
    for (const Matrix& m : all)
        if (m.bytes() && !ar::device_resident(m.p, m.bytes(), device)) return AR_ERR_INVALID_ARG;
    return AR_OK;
}

// One call: what it was given, and its launches.
struct Call {
    const ar_output_loss_s* h;
    const ar_output_loss_args* a;
    cudaStream_t st;
    uint32_t n, width, vocab;
    bool grads, packed = false;
    // of the pass at hand: the gradients that it makes, the logits' gradients' planes, and the
    // tokens whose logits' gradients are kept
    bool to_hidden = false, to_weight = false;
    int planes = 1;
    uint64_t kept = 0;
    float c = 0.f;
    double t = 1.0;
    ar::Lists lists = {};
    ar::Counted rows = {};
    cudaError_t e = cudaSuccess;

    Call(const ar_output_loss_s* h_, const ar_output_loss_args* a_, cudaStream_t st_)
        : h(h_), a(a_), st(st_), n(static_cast<uint32_t>(a_->tokens)), width(static_cast<uint32_t>(h_->hidden)),
          vocab(static_cast<uint32_t>(h_->vocab)), grads(a_->grad_weight || a_->grad_hidden) {
        lists.ids = h->at<int32_t>(h->l.ids);
        lists.entropy = h->at<float>(h->l.entropy);
        lists.counted = h->at<uint32_t>(h->l.counted);
        lists.logits = h->at<float>(h->l.logits);
        lists.top = 1;
        rows.count = h->at<uint32_t>(h->l.count);
        rows.row = h->at<int32_t>(h->l.row);
        rows.factor = h->at<float>(h->l.factor);
    }

    // Places [r, ...) of the counted tokens' hidden states; of the kept logits' gradients.
    ar::Planes hidden(uint64_t r) const {
        return {h->at<uint16_t>(h->l.hidden) + r * h->l.pitch, h->l.rows * h->l.pitch, h->l.pitch, h->l.planes};
    }
    ar::Planes grad(uint64_t r) const {
        ar::Planes g = {h->at<uint16_t>(h->l.grad) + r % kept * h->l.wide, kept * h->l.wide, h->l.wide, planes};
        if (planes != h->l.planes) g.low = h->at<uint16_t>(h->l.z);  // a piece at a time: r is its first
        return g;
    }
    // TMA reads rows that start on 16-byte boundaries
    bool weight_as_is() const {
        return h->dtype == AR_BFLOAT16 && reinterpret_cast<uintptr_t>(a->weight) % 16 == 0 &&
               a->weight_stride % 8 == 0 && a->weight_stride < (1ull << 38);
    }
    // Vocabulary entries that are at hand at a time, [v0, v1) as planes: where they are, or packed.
    uint64_t entries() const { return weight_as_is() ? h->vocab : std::min(h->vocab, h->l.pack); }
    // All of them stay packed for the call.
    ar::Planes weight(uint64_t v0, uint64_t v1) {
        if (weight_as_is())
            return {static_cast<uint16_t*>(const_cast<void*>(a->weight)) + v0 * a->weight_stride, 0, a->weight_stride, 1};
        const ar::PackArgs p = pack_weight(v0, v1);
        if (!packed) run(ar::launch_pack(p, nullptr, st));
        packed = v0 == 0 && v1 == h->vocab;
        return p.out;
    }
    ar::PackArgs pack_weight(uint64_t v0, uint64_t v1) const {
        ar::PackArgs p = {};
        p.src = static_cast<const char*>(a->weight) + v0 * a->weight_stride * esize(h->dtype);
        p.stride = a->weight_stride;
        p.bf16 = h->dtype == AR_BFLOAT16;
        p.n = static_cast<uint32_t>(v1 - v0);
        p.width = width;
        p.out = {h->at<uint16_t>(h->l.weight), h->l.pack * h->l.pitch, h->l.pitch, h->l.planes};
        return p;
    }
    void run(cudaError_t next) {
        if (e == cudaSuccess) e = next;
    }

    uint32_t run_of(ar_dtype result, int planes_a) const {
        if (h->dtype == AR_FLOAT32) return kFloatRun;
        return result == AR_FLOAT32 ? (planes_a == 1 ? kExactRun : kPlanesRun) : kLongRun / planes_a;
    }

    // Of the counted tokens at places [r, r + m).
    ar::ProductArgs product(uint64_t r) const {
        ar::ProductArgs p = {};
        p.count = rows.count;
        p.base = static_cast<uint32_t>(r);
        p.out.factor = rows.factor;
        p.out.t = static_cast<float>(t);
        p.status = h->at<uint32_t>(h->l.status);
        return p;
    }

    // Whether the call is on few enough tokens for the kernels that read the weights
    // as they are, of eight tokens at a time.  Losses alone / with gradients in a captured
    // graph, us, those kernels against tiles:
    //   bf16 W                n = 2              n = 4              n = 5              n = 8
    //   4096 x 128000   208  730 : 304 1840  298  997 : 303 1843  485 1320 : 297 1834  545 1400 : 291 1841
    //   2048 x 50000     56  189 :  84  401   76  253 :  72  387  125  349 :  74  389  139  374 :  69  389
    //   1024 x 32000     23  104 :  35  149   30  125 :  31  147   47  160 :  31  148   51  167 :  31  150
    //   640 x 10007      15   43 :  21   66   18   54 :  23   66   27   68 :  23   66   29   72 :  21   66
    //   192 x 4001       12   25 :  17   31   14   29 :  17   31   15   33 :  17   33   17   35 :  17   33
    //   1023 x 32003     27  121 :  61  376   39  153 :  60  375   45  174 :  56  372   49  181 :  54  373
    //   float32 W             n = 8              n = 9              n = 16             n = 24
    //   4096 x 128000   653 1537 :1933 6525 1023 2930 :1934 6536 1303 3853 :1933 6540 1972 6185 :1934 6558
    //   2048 x 50000    146  378 : 358  848  223  688 : 358  849  286  909 : 359  848  426 1441 : 359  851
    //   1024 x 32000     52  190 : 135  309   87  334 : 135  309  110  427 : 135  310  162  664 : 136  312
    //   1024 x 4096      25   51 :  49   84   35   99 :  50   85   41  107 :  50   86   58  169 :  51   86
    //   192 x 4001       17   35 :  23   39   23   64 :  23   39   25   66 :  23   39   33   98 :  23   40
    // The tiles' float32 pays for packing the weights in planes, twice (for the logits and
    // for the gradient of hidden states) where they are packed in turn; their odd bf16 rows
    // for packing them at all.  More than eight tokens of float32 are taken in groups, each
    // of which reads the weights and adds to their gradient.
    bool few() const {
        const uint64_t bytes = static_cast<uint64_t>(vocab) * width * esize(h->dtype), mb = 1u << 20;
        if (n == 0) return false;
        if (h->dtype == AR_FLOAT32) {
            if (n <= 8) return true;
            return grads ? n <= 24 && entries() < vocab : n <= 16 && bytes >= 8 * mb;
        }
        if (n <= 2 || (n <= 8 && (!weight_as_is() || bytes < 4 * mb))) return true;
        return n <= 4 ? grads || bytes < 128 * mb : n <= 8 && grads && bytes >= 128 * mb;
    }

    ar::FewArgs few_args(uint64_t r) const {
        ar::FewArgs f = {};
        f.x = a->hidden;
        f.w = a->weight;
        f.x_stride = a->hidden_stride;
        f.w_stride = a->weight_stride;
        f.bf16 = h->dtype == AR_BFLOAT16;
        f.base = static_cast<uint32_t>(r);
        f.n = static_cast<uint32_t>(std::min<uint64_t>(n - r, ar::kFewTokens));
        f.width = width;
        f.vocab = vocab;
        f.rows = rows;
        f.c = c;
        f.lists = lists;
        f.stats = h->at<float2>(h->l.stats);
        f.stats_pitch = h->l.wide / ar::kFewColumns;
        if (grads) f.z = h->at<float>(h->l.z);
        f.z_pitch = h->l.wide;
        return f;
    }

    // A few tokens' logits' gradients: 24 bits of them, whatever the inputs' type.
    ar::Planes few_grad() const {
        static_assert(ar::kFewTokens * ar::kMaxPlanes <= ar::kLossTile, "they fit the tiles' place");
        return {h->at<uint16_t>(h->l.grad), ar::kFewTokens * h->l.wide, h->l.wide, ar::kMaxPlanes};
    }

    ar::FewArgs few_gradients(ar::FewArgs f) const {
        f.g = few_grad();
        f.t = static_cast<float>(t);
        f.grad_x = a->grad_hidden;
        f.grad_w = a->grad_weight;
        f.grad_x_stride = a->grad_hidden_stride;
        f.grad_w_stride = a->grad_weight_stride;
        f.grad_x_bf16 = a->grad_hidden_dtype == AR_BFLOAT16;
        f.grad_w_bf16 = a->grad_weight_dtype == AR_BFLOAT16;
        f.accumulate = a->accumulate;
        f.parts = h->at<float>(h->l.part);
        f.room = h->l.part_room;
        return f;
    }

    // Logits, losses and gradients of a few tokens; the last group's CTAs write the record.
    void few_tokens() {
        for (uint64_t r = 0; r < n; r += ar::kFewTokens) {
            const ar::FewArgs f = few_args(r);
            run(ar::launch_few_logits(f, st));
            join(r, f.n, f.stats_pitch, ar::kFewColumns, 1);
            if (!grads) continue;
            const bool last = r + f.n >= n;
            run(ar::launch_few_gradients(few_gradients(f), {h->at<float>(h->l.loss), rows, last ? a->result : nullptr}, st));
        }
    }

    // Logits and losses of a piece, and the logits' gradients.
    void losses(uint64_t r, uint32_t m) {
        const uint64_t pitch = h->l.wide / ar::kStatColumns;
        for (uint64_t v = 0; v < h->vocab; v += entries()) {
            const uint64_t end = std::min(h->vocab, v + entries());
            ar::ProductArgs p = product(r);
            p.a = {hidden(r), false, m, h->hidden};
            p.b = {weight(v, end), false, end - v, h->hidden};
            p.m = m;
            p.count_m = 1;
            p.n = static_cast<uint32_t>(end - v);
            p.k = width;
            p.run = run_of(AR_FLOAT32, 1);
            p.logit.c = c;
            p.logit.v0 = static_cast<uint32_t>(v);
            p.logit.lists = lists;
            p.logit.row = rows.row + r;
            p.logit.stats = h->at<float2>(h->l.stats) + v / ar::kStatColumns;
            p.logit.stats_pitch = pitch;
            if (grads) p.logit.z = h->at<float>(h->l.z) + v;
            p.logit.at_ids = !grads || planes != h->l.planes;
            p.logit.z_pitch = h->l.wide;
            run(ar::launch_logits(p, st));
        }
        join(r, m, pitch, ar::kStatColumns, 64);  // whole blocks of products
    }

    void join(uint64_t r, uint32_t m, uint64_t pitch, uint32_t columns, uint32_t round) {
        ar::JoinArgs j = {};
        j.stats = h->at<float2>(h->l.stats);
        j.pitch = pitch;
        j.parts = static_cast<uint32_t>(up(h->vocab, columns) / columns);
        j.round = round;
        j.base = static_cast<uint32_t>(r);
        j.n = m;
        j.c = c;
        j.t2 = static_cast<float>(t * t);
        j.lists = lists;
        j.rows = rows;
        j.losses = a->losses;
        if (grads) {
            j.z = h->at<float>(h->l.z);
            j.z_pitch = h->l.wide;
            j.vocab = vocab;
            j.loss = h->at<float>(h->l.loss) + r;
            j.g = columns == ar::kFewColumns ? few_grad() : grad(r);
            run(ar::launch_grad(j, st));
        } else {
            j.sums = h->at<double>(h->l.sums);
            j.bad = h->at<uint32_t>(h->l.bad);
            j.ticket = h->at<uint32_t>(h->l.ticket);
            j.tickets = (n + ar::kJoinRows - 1) / ar::kJoinRows;
            j.result = a->result;
            run(ar::launch_join(j, st));
        }
    }

    // The last tokens' product goes to the caller, with the sum of those before; in
    // float32 every product does.
    ar::ProductArgs grad_weight(uint64_t r, uint32_t m, bool last) const {
        ar::ProductArgs p = product(r);
        p.a = {grad(r), true, m, h->vocab};
        p.b = {hidden(r), true, m, h->hidden};
        p.m = vocab;
        p.n = width;
        p.k = m;
        p.count_k = 1;
        p.run = run_of(a->grad_weight_dtype, planes);
        p.out.out = a->grad_weight;
        p.out.stride = a->grad_weight_stride;
        p.out.bf16 = a->grad_weight_dtype == AR_BFLOAT16;
        p.out.accumulate = a->accumulate || (!p.out.bf16 && r > 0);
        p.out.sum_pitch = p.out.part_pitch = h->l.sum_pitch;
        if (p.out.bf16 && r > 0) p.out.add = h->at<float>(h->l.sum);
        if (p.out.bf16 && !last) p.out.sum = h->at<float>(h->l.sum);
        if (!p.out.add && !p.out.sum) p.out.parts = h->at<float>(h->l.part);
        return p;
    }

    // By vocabulary entries [v, end), which are all of them, or packed in turn and
    // summed up in the parts' memory.
    ar::ProductArgs grad_hidden(uint64_t r, uint32_t m, uint64_t v, uint64_t end) {
        ar::ProductArgs p = product(r);
        ar::Planes g = grad(r);
        g.p += v;
        if (g.low) g.low += 2 * v;  // v is of whole tiles
        p.a = {g, false, m, end - v};
        p.b = {weight(v, end), true, end - v, h->hidden};
        p.m = m;
        p.count_m = 1;
        p.n = width;
        p.k = static_cast<uint32_t>(end - v);
        p.run = run_of(a->grad_hidden_dtype, planes);
        p.out.out = a->grad_hidden;
        p.out.stride = a->grad_hidden_stride;
        p.out.bf16 = a->grad_hidden_dtype == AR_BFLOAT16;
        p.out.accumulate = a->accumulate;
        p.out.row = rows.row + r;
        p.out.sum_pitch = p.out.part_pitch = h->l.sum_pitch;
        if (v > 0) p.out.add = h->at<float>(h->l.part);
        if (end < h->vocab) p.out.sum = h->at<float>(h->l.part);
        if (!p.out.add && !p.out.sum) p.out.parts = h->at<float>(h->l.part);
        return p;
    }

    // Both gradients of the kept tokens, in one launch but for packed weights.
    void gradients(uint64_t r, uint32_t m, bool last) {
        ar::RecordArgs record = {h->at<float>(h->l.loss), rows, last && m > 0 ? a->result : nullptr};
        ar::ProductArgs p[2];
        int k = 0;
        if (to_hidden && m > 0) {
            uint64_t v = 0;
            for (; v + entries() < h->vocab; v += entries()) {
                const ar::ProductArgs q = grad_hidden(r, m, v, v + entries());
                run(ar::launch_products(&q, 1, h->l.part_room, {}, st));
            }
            p[k++] = grad_hidden(r, m, v, h->vocab);
        }
        if (to_weight) p[k++] = grad_weight(r, m, last);
        run(ar::launch_products(p, k, h->l.part_room, record, st));
    }

    // Losses and the gradients asked for.  Of bf16 inputs logits' gradients are float32's 24
    // bits in three planes where a result is float32, and of a few tokens, whose products
    // cost what reading the weights does; else bf16, rounded once.  The planes that the
    // workspace has no place for take that of the piece's logits, so pieces are not kept:
    // the gradient of weights is summed piece by piece.  4096 tokens of 2048 x 50001 take
    // 3.76 ms for both gradients in float32, 7e-7 off the definition; of rounded logits'
    // gradients they took 1.84 and were 1.1e-3 off.
    void pass(bool hidden, bool weight) {
        to_hidden = hidden;
        to_weight = weight;
        const bool exact = (hidden && a->grad_hidden_dtype == AR_FLOAT32) || (weight && a->grad_weight_dtype == AR_FLOAT32);
        planes = exact || (grads && n <= ar::kFewTokens) ? ar::kMaxPlanes : h->l.planes;
        kept = h->l.kept;
        if (planes != h->l.planes) kept = h->l.piece;
        for (uint64_t first = 0; first < n || first == 0; first += kept) {
            const uint32_t all = static_cast<uint32_t>(std::min<uint64_t>(n - first, kept));
            for (uint64_t at = first; at < first + all; at += h->l.piece)
                losses(at, static_cast<uint32_t>(std::min<uint64_t>(first + all - at, h->l.piece)));
            if (to_weight || (to_hidden && all > 0)) gradients(first, all, first + kept >= n);
        }
    }

    // Everything after the lists: the tokens that count, then in pieces of them
    // logits, losses and gradients, and the record.
    ar_status finish(ar::RowsArgs r, double temperature) {
        t = temperature;
        c = static_cast<float>(1.4426950408889634 / t);
        r.n = n;
        r.vocab = vocab;
        r.scale = a->scale;
        r.mean = a->reduction == AR_LOSS_MEAN;
        r.lists = lists;
        r.rows = rows;
        r.result = a->result;
        r.ticket = h->at<uint32_t>(h->l.ticket);
        if (few()) {
            r.losses = a->losses;
            r.grad = a->accumulate ? nullptr : a->grad_hidden;
            r.grad_stride = a->grad_hidden_stride;
            r.grad_bf16 = a->grad_hidden_dtype == AR_BFLOAT16;
            r.width = width;
        }
        run(ar::launch_rows(r, st));
        if (few()) {
            few_tokens();
            return cuda_status(e);
        }
        if (n > 0) {
            ar::PackArgs p = {};
            p.src = a->hidden;
            p.stride = a->hidden_stride;
            p.bf16 = h->dtype == AR_BFLOAT16;
            p.n = n;
            p.width = width;
            p.rows = rows;
            p.out = hidden(0);
            p.counted = lists.counted;
            p.losses = a->losses;
            p.grad = a->accumulate ? nullptr : a->grad_hidden;
            p.grad_stride = a->grad_hidden_stride;
            p.grad_bf16 = a->grad_hidden_dtype == AR_BFLOAT16;
            // with the weights, where all of them are packed at a time
            packed = !weight_as_is() && entries() == h->vocab;
            const ar::PackArgs w = packed ? pack_weight(0, h->vocab) : ar::PackArgs{};
            run(ar::launch_pack(p, packed ? &w : nullptr, st));
        }
        // one gradient in each type: two passes, so that the float32 one is of float32 and the
        // bf16 one's sums need no more runs
        if (grads && h->dtype == AR_BFLOAT16 && n > ar::kFewTokens && a->grad_hidden && a->grad_weight &&
            a->grad_hidden_dtype != a->grad_weight_dtype) {
            pass(true, false);
            pass(false, true);
        } else {
            pass(a->grad_hidden, a->grad_weight);
        }
        return cuda_status(e);
    }
};

// What both losses' arguments have to be; `more`: the call's own inputs.
ar_status check_args(const ar_output_loss_s* h, const ar_output_loss_args* a, std::vector<Matrix> more) {
    if (!h || !a || a->tokens > h->tokens || !on_device(h->device)) return AR_ERR_INVALID_ARG;
    if (!float_normal(a->scale) || (a->reduction != AR_LOSS_MEAN && a->reduction != AR_LOSS_SUM)) return AR_ERR_INVALID_ARG;
    if (!h->gradients && (a->grad_hidden || a->grad_weight)) return AR_ERR_INVALID_ARG;
    if (a->grad_hidden && a->grad_hidden_dtype != h->dtype && a->grad_hidden_dtype != AR_FLOAT32) return AR_ERR_INVALID_ARG;
    if (a->grad_weight && a->grad_weight_dtype != h->dtype && a->grad_weight_dtype != AR_FLOAT32) return AR_ERR_INVALID_ARG;
    const int es = esize(h->dtype);
    more.push_back({a->hidden, a->tokens, h->hidden, a->hidden_stride, es});
    more.push_back({a->weight, h->vocab, h->hidden, a->weight_stride, es});
    std::vector<Matrix> out = {{a->result, 1, 4, 4, 4}};
    if (a->losses) out.push_back({a->losses, 1, a->tokens, a->tokens, 4});
    if (a->grad_hidden)
        out.push_back({a->grad_hidden, a->tokens, h->hidden, a->grad_hidden_stride, esize(a->grad_hidden_dtype)});
    if (a->grad_weight)
        out.push_back({a->grad_weight, h->vocab, h->hidden, a->grad_weight_stride, esize(a->grad_weight_dtype)});
    return check_matrices(more, out, h->device);
}

}  // namespace

extern "C" {

ar_status ar_output_loss_layout(uint64_t tokens, uint64_t hidden, uint64_t vocab, ar_dtype dtype, int top,
                                uint64_t piece, int gradients, ar_output_loss_info* info) {
    if (!info) return AR_ERR_INVALID_ARG;
    std::memset(info, 0, sizeof(*info));
    Layout l;
    const ar_status s = make_layout(tokens, hidden, vocab, dtype, top, piece, gradients, l);
    if (s != AR_OK) return s;
    info->tokens = tokens;
    info->hidden = hidden;
    info->vocab = vocab;
    info->top = top;
    info->piece = l.piece;
    info->pieces = static_cast<int>(l.pieces);
    info->workspace_bytes = l.bytes;
    info->tiling_ok = l.piece % ar::kLossTile == 0 && l.piece * l.pieces >= tokens && l.piece * (l.pieces - 1) < l.rows;
    return AR_OK;
}

ar_status ar_output_loss_create(uint64_t tokens, uint64_t hidden, uint64_t vocab, ar_dtype dtype, int top,
                                uint64_t piece, int gradients, ar_output_loss_t* out) {
    ar::TraceRange trace("ar_output_loss_create");
    if (!out) return AR_ERR_INVALID_ARG;
    *out = nullptr;
    Layout l;
    const ar_status s = make_layout(tokens, hidden, vocab, dtype, top, piece, gradients, l);
    if (s != AR_OK) return s;
    ar_output_loss_s* h = new (std::nothrow) ar_output_loss_s();
    if (!h) return AR_ERR_NOMEM;
    h->tokens = tokens;
    h->hidden = hidden;
    h->vocab = vocab;
    h->dtype = dtype;
    h->top = top;
    h->gradients = gradients != 0;
    h->l = l;
    cudaError_t e = cudaGetDevice(&h->device);
    if (e == cudaSuccess) e = ar::prepare_products();
    if (e == cudaSuccess) e = cudaMalloc(&h->dev, l.bytes);
    // in place on return: the calls may run on streams that do not wait for this one
    if (e == cudaSuccess) e = cudaMemset(h->dev, 0, l.sums);
    if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
    if (e != cudaSuccess) {
        delete h;
        return cuda_status(e);
    }
    *out = h;
    return AR_OK;
}

ar_status ar_output_loss_query(ar_output_loss_t h, ar_output_loss_info* info) {
    if (!h || !info) return AR_ERR_INVALID_ARG;
    return ar_output_loss_layout(h->tokens, h->hidden, h->vocab, h->dtype, h->top, h->l.piece, h->gradients, info);
}

ar_status ar_output_loss_destroy(ar_output_loss_t h) {
    if (!h) return AR_ERR_INVALID_ARG;
    int now = -1;
    cudaError_t e = cudaGetDevice(&now);
    const bool other = e == cudaSuccess && now != h->device;
    if (other) e = cudaSetDevice(h->device);
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    delete h;
    if (other) cudaSetDevice(now);
    return cuda_status(e);
}

ar_status ar_output_loss_check(ar_output_loss_t h) {
    if (!h || !on_device(h->device)) return AR_ERR_INVALID_ARG;
    uint32_t word = 0;
    cudaError_t e = cudaDeviceSynchronize();
    if (e == cudaSuccess) e = cudaMemcpy(&word, h->at<uint32_t>(h->l.status), 4, cudaMemcpyDeviceToHost);
    if (e == cudaSuccess && word) e = cudaMemset(h->at<uint32_t>(h->l.status), 0, 4);
    if (e == cudaSuccess && word) e = cudaStreamSynchronize(nullptr);
    if (e != cudaSuccess) return cuda_status(e);
    return word ? AR_ERR_TIMEOUT : AR_OK;
}

ar_status ar_output_cross_entropy(ar_output_loss_t h, const ar_output_loss_args* args, const void* targets,
                                  int target_bytes, int64_t ignore_index, void* stream) {
    ar::TraceRange trace("ar_output_cross_entropy");
    if (!h || !args || (target_bytes != 4 && target_bytes != 8)) return AR_ERR_INVALID_ARG;
    try {
        const ar_status s = check_args(h, args, {{targets, 1, args->tokens, args->tokens, target_bytes}});
        if (s != AR_OK) return s;
        Call call(h, args, static_cast<cudaStream_t>(stream));
        ar::RowsArgs r = {};
        r.targets = targets;
        r.target_bytes = target_bytes;
        r.ignore = ignore_index;
        return call.finish(r, 1.0);
    } catch (const std::bad_alloc&) {
        return AR_ERR_NOMEM;
    }
}

ar_status ar_output_distill(ar_output_loss_t h, const ar_output_loss_args* args, const void* ids, int id_bytes,
                            uint64_t ids_stride, const void* logits, ar_dtype logit_dtype, uint64_t logits_stride,
                            int k, double temperature, void* stream) {
    ar::TraceRange trace("ar_output_distill");
    if (!h || !args || (id_bytes != 4 && id_bytes != 8) || !float_dtype(logit_dtype)) return AR_ERR_INVALID_ARG;
    if (k < 1 || k > h->top || !float_normal(temperature) || !float_normal(1.0 / temperature) ||
        !float_normal(temperature * temperature))
        return AR_ERR_INVALID_ARG;
    try {
        const uint64_t width = static_cast<uint64_t>(k);
        const ar_status s = check_args(h, args, {{ids, args->tokens, width, ids_stride, id_bytes},
                                                 {logits, args->tokens, width, logits_stride, esize(logit_dtype)}});
        if (s != AR_OK) return s;
        Call call(h, args, static_cast<cudaStream_t>(stream));
        call.lists.top = k;
        call.lists.shares = h->at<float>(h->l.shares);
        if (args->tokens > 0) {
            ar::TeacherArgs t = {};
            t.ids = ids;
            t.logits = logits;
            t.ids_stride = ids_stride;
            t.logits_stride = logits_stride;
            t.id_bytes = id_bytes;
            t.logits_bf16 = logit_dtype == AR_BFLOAT16;
            t.k = k;
            t.inv_t = static_cast<float>(1.0 / temperature);
            t.n = call.n;
            t.vocab = static_cast<uint32_t>(h->vocab);
            t.lists = call.lists;
            call.run(ar::launch_teacher(t, call.st));
        }
        return call.finish({}, temperature);
    } catch (const std::bad_alloc&) {
        return AR_ERR_NOMEM;
    }
}

}  // extern "C"
