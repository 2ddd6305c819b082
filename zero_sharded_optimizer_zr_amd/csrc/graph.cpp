// Captured steps: a sequence of library calls recorded once on a stream as a
// HIP graph and replayed as one launch.  Small shards are launch-bound (the
// tiny MLP's four-call step moves 14 MB in 40 us of launches), and a training
// loop repeats the same calls on the same buffers every step; what changes is
// the AdamW step number t (its bias corrections) and possibly the learning
// rate.  Those enter the AdamW-family kernels as one by-value argument
// (AdamWScalars), so the graph keeps, for every captured kernel node that
// takes it, the node and its argument list, and zr_graph_set_adamw rewrites
// that one argument on the instantiated graph (hipGraphExecKernelNodeSetParams)
// before the next replay.  A captured gradient norm holds the step's grad_scale
// too: where it was captured with a step's, it is rewritten with it, or the step
// would be bounded by the norm at the old scale.  Everything else -- buffers, sizes, layout
// descriptors, the fp16 loss-scale record -- is fixed at capture.
#include <algorithm>
#include <new>
#include <vector>

#include "clip.hpp"

struct zr_graph {
    hipGraph_t graph = nullptr;
    hipGraphExec_t exec = nullptr;
    struct Node {
        hipGraphNode_t node;
        hipKernelNodeParams params;
        std::vector<void *> args;  // the captured argument pointers; args[index] is replaced
        int index;
    };
    std::vector<Node> adamw;
    std::vector<Node> norms;  // those captured with the grad_scale of one of `adamw`
    int kernels = 0;
};

namespace zr {
namespace {

std::vector<ScalarSlot> all_slots()
{
    std::vector<ScalarSlot> v(4 * kMaxScalarSlots);
    int k = adamw_scalar_slots(v.data());
    k += fused_scalar_slots(v.data() + k);
    k += fp16_scalar_slots(v.data() + k);
    k += clip_scalar_slots(v.data() + k);
    v.resize(k);
    return v;
}

std::vector<ScalarSlot> norm_slots()
{
    std::vector<ScalarSlot> v(kMaxScalarSlots);
    v.resize(norm_finish_slots(v.data()));
    return v;
}

// Adds the node to `nodes` if its kernel is one of the slots'.  False if it is and has
// no argument list.
bool keep_node(const std::vector<ScalarSlot> &slots, hipGraphNode_t node, const hipKernelNodeParams &p,
               std::vector<zr_graph::Node> *nodes)
{
    for (const ScalarSlot &sl : slots) {
        if (sl.func != p.func)
            continue;
        if (!p.kernelParams)
            return false;
        nodes->push_back({node, p, std::vector<void *>(p.kernelParams, p.kernelParams + sl.nargs), sl.index});
        break;
    }
    return true;
}

// The node's argument becomes `value` in the following launches (the call copies it).
hipError_t set_argument(hipGraphExec_t exec, const zr_graph::Node &n, void *value)
{
    std::vector<void *> args = n.args;
    args[n.index] = value;
    hipKernelNodeParams p = n.params;
    p.kernelParams = args.data();
    p.extra = nullptr;
    return hipGraphExecKernelNodeSetParams(exec, n.node, &p);
}

zr_status hip_fail(const char *who, const char *what, hipError_t e)
{
    return fail(ZR_EHIP, "%s: %s: %s", who, what, hipGetErrorString(e));
}

}  // namespace
}  // namespace zr

using namespace zr;

extern "C" zr_status zr_graph_capture_begin(void *stream)
{
    clear_error();
    if (!stream)
        return fail(ZR_EINVAL, "zr_graph_capture_begin: the null stream cannot be captured");
    hipError_t e = hipStreamBeginCapture(static_cast<hipStream_t>(stream), hipStreamCaptureModeThreadLocal);
    return e == hipSuccess ? ZR_OK : hip_fail("zr_graph_capture_begin", "hipStreamBeginCapture", e);
}

extern "C" zr_status zr_graph_capture_end(void *stream, zr_graph **out)
{
    clear_error();
    const char *who = "zr_graph_capture_end";
    if (!stream || !out)
        return fail(ZR_EINVAL, "%s: NULL stream or out", who);
    *out = nullptr;
    auto *g = new (std::nothrow) zr_graph;
    if (!g) {
        hipGraph_t dropped = nullptr;
        if (hipStreamEndCapture(static_cast<hipStream_t>(stream), &dropped) == hipSuccess && dropped)
            (void)hipGraphDestroy(dropped);
        return fail(ZR_ENOMEM, "%s: out of host memory", who);
    }
    auto bail = [&](zr_status s) {
        zr_graph_destroy(g);
        return s;
    };
    hipError_t e = hipStreamEndCapture(static_cast<hipStream_t>(stream), &g->graph);
    if (e != hipSuccess)
        return bail(hip_fail(who, "hipStreamEndCapture", e));
    if (!g->graph)
        return bail(fail(ZR_EINVAL, "%s: nothing was captured", who));
    size_t count = 0;
    if ((e = hipGraphGetNodes(g->graph, nullptr, &count)) != hipSuccess)
        return bail(hip_fail(who, "hipGraphGetNodes", e));
    std::vector<hipGraphNode_t> nodes(count);
    if (count && (e = hipGraphGetNodes(g->graph, nodes.data(), &count)) != hipSuccess)
        return bail(hip_fail(who, "hipGraphGetNodes", e));
    const std::vector<ScalarSlot> slots = all_slots(), norms = norm_slots();
    for (hipGraphNode_t n : nodes) {
        hipGraphNodeType type;
        if ((e = hipGraphNodeGetType(n, &type)) != hipSuccess)
            return bail(hip_fail(who, "hipGraphNodeGetType", e));
        if (type != hipGraphNodeTypeKernel)
            continue;
        ++g->kernels;
        hipKernelNodeParams p{};
        if ((e = hipGraphKernelNodeGetParams(n, &p)) != hipSuccess)
            return bail(hip_fail(who, "hipGraphKernelNodeGetParams", e));
        if (!keep_node(slots, n, p, &g->adamw) || !keep_node(norms, n, p, &g->norms))
            return bail(fail(ZR_EHIP, "%s: a captured AdamW or norm node has no argument list", who));
    }
    g->norms.erase(std::remove_if(g->norms.begin(), g->norms.end(), [&](const zr_graph::Node &n) {
        const double scale = static_cast<const NormFinish *>(n.args[n.index])->grad_scale;
        return std::none_of(g->adamw.begin(), g->adamw.end(), [&](const zr_graph::Node &a) {
            return static_cast<const AdamWScalars *>(a.args[a.index])->grad_scale == scale;
        });
    }), g->norms.end());
    if ((e = hipGraphInstantiate(&g->exec, g->graph, nullptr, nullptr, 0)) != hipSuccess)
        return bail(hip_fail(who, "hipGraphInstantiate", e));
    *out = g;
    return ZR_OK;
}

extern "C" zr_status zr_graph_info(const zr_graph *g, int32_t *kernels, int32_t *adamw_nodes)
{
    clear_error();
    if (!g)
        return fail(ZR_EINVAL, "zr_graph_info: graph is NULL");
    if (kernels)
        *kernels = g->kernels;
    if (adamw_nodes)
        *adamw_nodes = (int32_t)g->adamw.size();
    return ZR_OK;
}

extern "C" zr_status zr_graph_set_adamw(zr_graph *g, const zr_adamw_hparams *hp)
{
    clear_error();
    const char *who = "zr_graph_set_adamw";
    if (!g)
        return fail(ZR_EINVAL, "%s: graph is NULL", who);
    zr_status st = check_adamw_hparams(who, hp);
    if (st != ZR_OK)
        return st;
    AdamWScalars s = adamw_scalars(*hp);
    for (const auto &a : g->adamw) {
        const hipError_t e = set_argument(g->exec, a, &s);
        if (e != hipSuccess)
            return hip_fail(who, "hipGraphExecKernelNodeSetParams", e);
    }
    for (const auto &n : g->norms) {
        NormFinish f = *static_cast<const NormFinish *>(n.args[n.index]);
        f.grad_scale = hp->grad_scale;
        const hipError_t e = set_argument(g->exec, n, &f);
        if (e != hipSuccess)
            return hip_fail(who, "hipGraphExecKernelNodeSetParams", e);
    }
    return ZR_OK;
}

extern "C" zr_status zr_graph_launch(zr_graph *g, void *stream)
{
    clear_error();
    if (!g)
        return fail(ZR_EINVAL, "zr_graph_launch: graph is NULL");
    hipError_t e = hipGraphLaunch(g->exec, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ZR_OK : hip_fail("zr_graph_launch", "hipGraphLaunch", e);
}

extern "C" void zr_graph_destroy(zr_graph *g)
{
    if (!g)
        return;
    if (g->exec)
        (void)hipGraphExecDestroy(g->exec);
    if (g->graph)
        (void)hipGraphDestroy(g->graph);
    delete g;
}
