"""GPU time of calls that are compared with one another: captured, many a
graph, and timed in turns."""
import torch


def in_turns(*calls, each=20, rounds=7):
    """Median microseconds of a call of each, warm."""
    graphs = []
    for call in calls:
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(each):
                call()
        graphs.append(g)
    took = [[] for _ in calls]
    for r in range(rounds + 1):
        for g, t in zip(graphs, took):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            g.replay()
            b.record()
            torch.cuda.synchronize()
            if r:
                t.append(a.elapsed_time(b) * 1e3 / each)
    return [sorted(t)[rounds // 2] for t in took]
